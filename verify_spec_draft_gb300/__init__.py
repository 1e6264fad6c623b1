"""GB300 (sm_103a) hot path of block speculative decoding: Python binding.

The compute lives in ``libspecgb300.so`` (CUDA kernels behind the C ABI declared in
``include/spec.h``).  This module only marshals arguments: it checks tensor dtypes,
devices and shapes, allocates outputs and workspaces with PyTorch, and passes raw
device pointers and the current CUDA stream to the library.  There is no CPU or
PyTorch fallback: every call fails loudly if the library is not built.

    import verify_spec_draft_gb300 as vsd
    vsd.load()                                   # after vsd.build.build()
    out = vsd.draft_block(logits, anchor, U, Wt, temperature=0)
    res = vsd.verify(target, None, out["tokens"], temperature=0)
    tv  = vsd.e2etv(target_rows, draft_rows, n_branches, Wb)
"""

import contextlib
import ctypes
import os

from . import build as _build

OK = 0
STATUS = {
    0: "SPEC_OK", 1: "SPEC_ERR_INVALID_ARG", 2: "SPEC_ERR_SHAPE", 3: "SPEC_ERR_DTYPE",
    4: "SPEC_ERR_ALIGN", 5: "SPEC_ERR_CUDA", 6: "SPEC_ERR_TIMEOUT", 7: "SPEC_ERR_NONFINITE",
    8: "SPEC_ERR_TOKEN", 9: "SPEC_ERR_WORKSPACE",
}
F32, BF16 = 0, 1
OP_DRAFT, OP_VERIFY, OP_E2ETV, OP_DRAFT_VERIFY, OP_BRANCH_PLAN, OP_VERIFY_TOPK, OP_TREE_VERIFY, OP_DRAFT_TOPK = (
    0, 1, 2, 3, 4, 5, 6, 7)
OP_PROCESS_LOGITS, OP_TOP_LOGITS, OP_DISTILL = 9, 10, 11
OP_POLICY_LOSS, OP_MARKOV_GRAD, OP_ADAMW = 12, 13, 14
DEV_TIMEOUT, DEV_NONFINITE, DEV_TOKEN = 1, 2, 4

# C signatures of include/spec.h, as ctypes types
_vp, _i32, _sz, _u32p = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.POINTER(ctypes.c_uint32)
SIGNATURES = {
    "spec_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32, _i32]),
    "spec_workspace_init": (_i32, [_vp, _sz, _vp]),
    "spec_get_device_status": (_i32, [_vp, _vp, _u32p]),
    "spec_status_string": (ctypes.c_char_p, [_i32]),
    "spec_last_cuda_error": (_i32, []),
    "spec_last_cuda_error_string": (ctypes.c_char_p, []),
    "spec_draft_block": (_i32, [_vp, _i32, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _vp,
                                _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "spec_verify": (_i32, [_vp, _i32, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _vp,
                           _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "spec_e2etv": (_i32, [_vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "spec_verify_noalloc": (_i32, [_vp, _i32, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _vp,
                                   _vp, _vp, _vp, _vp, _vp]),
    "spec_draft_verify": (_i32, [_vp, _i32, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _i32,
                                 _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "spec_verify_budget": (_i32, [_vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp]),
    "spec_verify_topk": (_i32, [_vp, _i32, _vp, _i32, _vp, _i32, _i32, _i32, _i32, ctypes.c_double, _vp, _vp, _vp,
                                _vp, _vp, _vp, _sz, _vp]),
    "spec_e2etv_shard": (_i32, [_vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "spec_branch_plan": (_i32, [_vp, _vp, _i32, _i32, _i32, _i32, ctypes.c_uint64, _vp, _vp, _vp, _vp,
                                _vp, _sz, _vp]),
    "spec_tree_select": (_i32, [_vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp]),
    "spec_draft_block_topk": (_i32, [_vp, _i32, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, ctypes.c_double,
                                     _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "spec_tree_verify": (_i32, [_vp, _i32, _vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "spec_process_logits": (_i32, [_vp, _i32, _i32, _i32, _i32, _i32, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                   _vp, _vp, _i32, _vp, _i32, _vp, _vp, _sz, _vp]),
    "spec_top_logits": (_i32, [_vp, _i32, _i32, _i32, _i32, _i32, ctypes.c_float, _vp, _vp, _vp, _vp, _vp, _sz,
                               _vp]),
    "spec_distill": (_i32, [_vp, _i32, _i32, _i32, _i32, _vp, _i32, _vp, _i32, _vp, _vp, ctypes.c_float, _vp, _vp,
                            _vp, _vp, _sz, _vp]),
    "spec_policy_loss": (_i32, [_vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, ctypes.c_float, ctypes.c_float,
                                ctypes.c_float, ctypes.c_float, _vp, _vp, _vp, _vp, _sz, _vp]),
    "spec_markov_grad": (_i32, [_vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _i32, _i32, _vp, _vp, _i32,
                                _vp, _sz, _vp]),
    "spec_adamw": (_i32, [_vp, _i32, _vp, ctypes.c_double, ctypes.c_double, ctypes.c_double, ctypes.c_double,
                          ctypes.c_double, _vp, ctypes.c_uint64, _vp, _sz, _vp]),
}


class AdamwTensor(ctypes.Structure):
    """spec_adamw_tensor of include/spec.h."""
    _fields_ = [(name, ctypes.c_void_p) for name in ("param", "master", "grad", "m", "v", "m_scale", "v_scale")] + [
        ("n", ctypes.c_int64), ("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32),
        ("state_bits", ctypes.c_int32), ("pad", ctypes.c_int32)]


ADAMW_BLOCK = 128   # entries that share an 8-bit state's scale
_STATE = ("master", "m", "v", "m_scale", "v_scale")
_lib = None


class SpecError(RuntimeError):
    def __init__(self, code, what):
        msg = f"{what}: {STATUS.get(code, code)} ({status_string(code)})"
        if code == 5 and _lib is not None:
            msg += f" [cuda error {_lib.spec_last_cuda_error()}: {_lib.spec_last_cuda_error_string().decode()}]"
        super().__init__(msg)
        self.code = code


def library_path():
    return _build.LIB


def load(path=None):
    """Load the compiled library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"libspecgb300.so not found at {path}: run verify_spec_draft_gb300.build.build() "
                           "(or __graft_entry__.build()) first; there is no fallback implementation")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def status_string(code):
    if _lib is None:
        return STATUS.get(code, "unknown")
    return _lib.spec_status_string(code).decode()


def _check(code, what):
    if code != OK:
        raise SpecError(code, what)


# ---------------------------------------------------------------------------------
# tensor marshalling helpers (no arithmetic)
# ---------------------------------------------------------------------------------
def _torch():
    import torch
    return torch


def _dtype_code(t):
    torch = _torch()
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"logits/weights must be float32 or bfloat16, got {t.dtype}")


def _ptr(t):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _need(t, name, device=None, dtype=None, shape=None):
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _need_rows(t, name, device=None):
    """Like _need for logits rows [..., V] that may lie further apart than V entries:
    returns the row stride.  The leading dimensions must be evenly spaced."""
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    shape = t.shape
    if len(shape) < 2:
        raise ValueError(f"{name} must be at least [rows, V]")
    V, ld, rows, strides = shape[-1], 0, 1, t.stride()
    if strides[-1] == 1 and strides[-2] == V and (len(shape) == 2 or (len(shape) == 3 and strides[0] == shape[1] * V)):
        return V   # contiguous: nothing more to look at
    if V > 1 and strides[-1] != 1:
        raise ValueError(f"{name} must have its entries next to one another (stride 1)")
    for n, st in zip(reversed(shape[:-1]), reversed(strides[:-1])):
        if n == 1:
            continue
        if ld == 0:
            ld = st // rows if st % rows == 0 else 0
        if ld < V or st != rows * ld:
            raise ValueError(f"{name} must have evenly spaced rows at least V entries apart, got strides {strides}")
        rows *= n
    return ld or V


def _current_device():
    return _torch()._C._cuda_getDevice()


def _away(device, stream):
    """Whether `device`, the rows', is not the one that calls launch on: then the call is made
    again under it.  A caller's stream has to be one of its."""
    if stream is not None and stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the rows on {device}")
    return _current_device() != device.index


_INT_MAX = 2**31 - 1


def _need_ints(what, *sizes):
    """Sizes that the C interface takes as 32-bit numbers: ctypes would pass them modulo 2^32."""
    if max(sizes) > _INT_MAX:
        raise SpecError(2, f"{what}{sizes}")


def _addrs(device, names, tensors, dtypes, shapes):
    """The addresses of optional contiguous tensors (None for None), checked as _need does,
    which says what is wrong; one loop, since a call's checks are most of its host time."""
    index, out = device.index, []
    for name, t, dtype, shape in zip(names, tensors, dtypes, shapes):
        if t is None:
            out.append(None)
            continue
        if t.dtype is not dtype or t.get_device() != index or t.shape != shape or not t.is_contiguous():
            _need(t, name, device, dtype, shape)
        out.append(t.data_ptr())
    return out


def _need_out(out, device, **want):
    """The caller's outputs, checked as _need does; lse may be left out."""
    for name, (dtype, shape) in want.items():
        t = out.get(name)
        if t is not None or name != "lse":
            _need(t, name, device, dtype, shape)


def _ws_bytes(ws, device):
    """A workspace's size, which the library compares with what it needs."""
    if ws.get_device() != device.index:
        raise ValueError(f"the workspace is on {ws.device}, expected {device}")
    return ws.numel()


_HERE = contextlib.nullcontext()


def _made_on(stream):
    """What a call allocates belongs to the stream it runs on."""
    return _HERE if stream is None else _torch().cuda.stream(stream)


def _rows_like(t, ld):
    """Uninitialised rows of t's shape, dtype and row stride."""
    torch = _torch()
    V = t.shape[-1]
    if ld == V:
        return torch.empty_like(t, memory_format=torch.contiguous_format)
    return torch.empty((*t.shape[:-1], ld), dtype=t.dtype, device=t.device)[..., :V]


def _need_same_rows(t, name, like, ld):
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype is not like.dtype or t.shape != like.shape:
        raise ValueError(f"{name} must be {like.dtype} {tuple(like.shape)}, got {t.dtype} {tuple(t.shape)}")
    if _need_rows(t, name, like.device) != ld and t.numel() > t.shape[-1]:
        raise ValueError(f"{name} must have the row stride {ld}")
    return t


def _stream(stream=None):
    if stream is None:
        # the current stream's handle without building a Stream object (11 us a call)
        C = _torch()._C
        return ctypes.c_void_p(C._cuda_getCurrentRawStream(C._cuda_getDevice()))
    return ctypes.c_void_p(stream.cuda_stream)


def workspace_bytes(op, B, gamma, V, r=0):
    n = load().spec_workspace_bytes(op, B, gamma, V, r)
    if n == 0:
        raise SpecError(2, f"workspace_bytes(op={op}, B={B}, gamma={gamma}, V={V}, r={r})")
    return n


def workspace(op, B, gamma, V, r=0, device=None, stream=None):
    """Allocate a device workspace for one operation and zero it (spec_workspace_init).

    Calls of that operation and shape can reuse it as it is; zero it again (or take a
    new one) before a call with another operation or shape."""
    torch = _torch()
    n = workspace_bytes(op, B, gamma, V, r)
    ws = torch.empty(n, dtype=torch.uint8, device=device or torch.device("cuda"))
    _check(load().spec_workspace_init(_ptr(ws), n, _stream(stream)), "spec_workspace_init")
    return ws


def device_status(ws, stream=None):
    """Synchronise and return the raw SPEC_DEV_* flags of a workspace."""
    flags = ctypes.c_uint32(0)
    load().spec_get_device_status(_ptr(ws), _stream(stream), ctypes.byref(flags))
    return flags.value


# ---------------------------------------------------------------------------------
# the three operations
# ---------------------------------------------------------------------------------
def draft_block(logits, anchor, U=None, Wt=None, temperature=0, seeds=None, ws=None,
                qlogits=False, out=None, stream=None):
    """spec_draft_block.  logits [B, gamma, V] f32/bf16; anchor [B] int32; U, Wt [V, r]
    (same dtype) or None; seeds [B] int64 (uint64 bits) at T=1.  Returns a dict of
    device tensors: tokens, conf, qtok, passes and (if ``qlogits``) the float32 z rows."""
    torch = _torch()
    lib = load()
    _need(logits, "logits")
    dev = logits.device
    B, gamma, V = logits.shape
    _need(anchor, "anchor", dev, torch.int32, (B,))
    r = 0
    if U is not None:
        _need(U, "U", dev)
        _need(Wt, "Wt", dev, U.dtype, tuple(U.shape))
        if U.shape[0] != V:
            raise ValueError("U and Wt must have V rows")
        r = U.shape[1]
    wdt = _dtype_code(U) if U is not None else F32
    if temperature == 1:
        _need(seeds, "seeds", dev, torch.int64, (B,))
    if out is None:
        out = dict(
            tokens=torch.empty((B, gamma), dtype=torch.int32, device=dev),
            conf=torch.empty((B, gamma), dtype=torch.float32, device=dev),
            qtok=torch.empty((B, gamma), dtype=torch.float32, device=dev),
            passes=torch.zeros((1,), dtype=torch.int32, device=dev),
        )
        if qlogits:
            out["qlogits"] = torch.empty((B, gamma, V), dtype=torch.float32, device=dev)
    if ws is None:
        ws = workspace(OP_DRAFT, B, gamma, V, r, dev, stream)
    code = lib.spec_draft_block(
        _ptr(logits), _dtype_code(logits), _ptr(anchor), _ptr(U), _ptr(Wt), wdt, r, B, gamma, V,
        int(temperature), _ptr(seeds), _ptr(out["tokens"]), _ptr(out["conf"]), _ptr(out.get("qtok")),
        _ptr(out.get("qlogits")), _ptr(out.get("passes")), _ptr(ws), ws.numel(), _stream(stream))
    _check(code, "spec_draft_block")
    out["ws"] = ws
    return out


def verify(target, draft, tokens, temperature=0, seeds=None, ws=None, out=None, stream=None):
    """spec_verify.  target [B, gamma+1, V]; draft [B, gamma, V] (T=1, else None);
    tokens [B, gamma] int32; seeds [B] int64 at T=1.  Returns a dict of device tensors:
    n (accepted drafts), committed, bonus, near."""
    torch = _torch()
    lib = load()
    _need(target, "target")
    dev = target.device
    B, g1, V = target.shape
    gamma = g1 - 1
    _need(tokens, "tokens", dev, torch.int32, (B, gamma))
    ddt = F32
    if temperature == 1:
        _need(draft, "draft", dev, None, (B, gamma, V))
        ddt = _dtype_code(draft)
        _need(seeds, "seeds", dev, torch.int64, (B,))
    if out is None:
        out = dict(
            n=torch.empty((B,), dtype=torch.int32, device=dev),
            committed=torch.empty((B, gamma + 1), dtype=torch.int32, device=dev),
            bonus=torch.empty((B,), dtype=torch.int32, device=dev),
            near=torch.empty((B,), dtype=torch.int32, device=dev),
        )
    if ws is None:
        ws = workspace(OP_VERIFY, B, gamma, V, 0, dev, stream)
    code = lib.spec_verify(
        _ptr(target), _dtype_code(target), _ptr(draft if temperature == 1 else None), ddt, _ptr(tokens),
        B, gamma, V, int(temperature), _ptr(seeds), _ptr(out["n"]), _ptr(out["committed"]), _ptr(out["bonus"]),
        _ptr(out.get("near")), _ptr(ws), ws.numel(), _stream(stream))
    _check(code, "spec_verify")
    out["ws"] = ws
    return out


def draft_verify(logits, target, anchor, U=None, Wt=None, ws=None, out=None, stream=None):
    """spec_draft_verify (T=0).  logits [B, gamma, V]; target [B, gamma+1, V]; anchor [B]
    int32; U, Wt [V, r] or None.  Returns a dict of device tensors: the draft's tokens,
    conf, qtok, passes and verify's n, committed, bonus."""
    torch = _torch()
    lib = load()
    _need(logits, "logits")
    dev = logits.device
    B, gamma, V = logits.shape
    _need(target, "target", dev, None, (B, gamma + 1, V))
    _need(anchor, "anchor", dev, torch.int32, (B,))
    r = 0
    if U is not None:
        _need(U, "U", dev)
        _need(Wt, "Wt", dev, U.dtype, tuple(U.shape))
        if U.shape[0] != V:
            raise ValueError("U and Wt must have V rows")
        r = U.shape[1]
    wdt = _dtype_code(U) if U is not None else F32
    if out is None:
        out = dict(
            tokens=torch.empty((B, gamma), dtype=torch.int32, device=dev),
            conf=torch.empty((B, gamma), dtype=torch.float32, device=dev),
            qtok=torch.empty((B, gamma), dtype=torch.float32, device=dev),
            passes=torch.zeros((1,), dtype=torch.int32, device=dev),
            n=torch.empty((B,), dtype=torch.int32, device=dev),
            committed=torch.empty((B, gamma + 1), dtype=torch.int32, device=dev),
            bonus=torch.empty((B,), dtype=torch.int32, device=dev),
        )
    if ws is None:
        ws = workspace(OP_DRAFT_VERIFY, B, gamma, V, r, dev, stream)
    code = lib.spec_draft_verify(
        _ptr(logits), _dtype_code(logits), _ptr(anchor), _ptr(U), _ptr(Wt), wdt, r, B, gamma, V,
        _ptr(target), _dtype_code(target), _ptr(out["tokens"]), _ptr(out["conf"]), _ptr(out.get("qtok")),
        _ptr(out.get("passes")), _ptr(out["n"]), _ptr(out["committed"]), _ptr(out["bonus"]), _ptr(ws),
        ws.numel(), _stream(stream))
    _check(code, "spec_draft_verify")
    out["ws"] = ws
    return out


def verify_budget(conf, budget, cost=None, out=None, stream=None):
    """spec_verify_budget.  conf [B, gamma] float32 (spec_draft_block's conf); budget:
    most draft positions verified in all; cost: float32 [budget + 1] time per total, or
    None.  Returns a dict of device tensors: gamma [B] int32, expected [1] float32."""
    torch = _torch()
    lib = load()
    _need(conf, "conf", None, torch.float32)
    if conf.dim() != 2:
        raise ValueError("conf must be [B, gamma]")
    dev = conf.device
    B, gamma = conf.shape
    if cost is not None:
        _need(cost, "cost", dev, torch.float32, (int(budget) + 1,))
    if out is None:
        out = dict(gamma=torch.empty((B,), dtype=torch.int32, device=dev),
                   expected=torch.empty((1,), dtype=torch.float32, device=dev))
    code = lib.spec_verify_budget(_ptr(conf), B, gamma, int(budget), _ptr(cost), _ptr(out["gamma"]),
                                  _ptr(out.get("expected")), _stream(stream))
    _check(code, "spec_verify_budget")
    return out


def branch_plan(trunk, lengths, n_anchors, W, seed, ws=None, out=None, stream=None):
    """spec_branch_plan.  trunk int32 [n_refs, Lmax] reference tokens; lengths int32
    [n_refs].  Returns a dict of device tensors: anchors, anchor_tok [n_refs, n_anchors]
    and parent, position [n_refs, n_anchors * W] (int32)."""
    torch = _torch()
    lib = load()
    _need(trunk, "trunk", None, torch.int32)
    if trunk.dim() != 2:
        raise ValueError("trunk must be [n_refs, Lmax]")
    dev = trunk.device
    R, Lmax = trunk.shape
    _need(lengths, "lengths", dev, torch.int32, (R,))
    if out is None:
        out = dict(anchors=torch.empty((R, n_anchors), dtype=torch.int32, device=dev),
                   anchor_tok=torch.empty((R, n_anchors), dtype=torch.int32, device=dev),
                   parent=torch.empty((R, n_anchors * W), dtype=torch.int32, device=dev),
                   position=torch.empty((R, n_anchors * W), dtype=torch.int32, device=dev))
    if ws is None:
        ws = workspace(OP_BRANCH_PLAN, R, W, Lmax, 0, dev, stream)
    code = lib.spec_branch_plan(_ptr(trunk), _ptr(lengths), R, Lmax, int(n_anchors), int(W), int(seed),
                                _ptr(out["anchors"]), _ptr(out["anchor_tok"]), _ptr(out["parent"]),
                                _ptr(out["position"]), _ptr(ws), ws.numel(), _stream(stream))
    _check(code, "spec_branch_plan")
    out["ws"] = ws
    return out


def verify_topk(target, draft, tokens, top_k, top_p, seeds, ws=None, out=None, stream=None):
    """spec_verify_topk (T=1 against top-k / top-p filtered rows).  target [B, gamma+1, V]
    and draft [B, gamma, V] f32/bf16; tokens [B, gamma] int32; seeds [B] int64.  Returns
    a dict of device tensors: n [B], committed [B, gamma+1], bonus [B], near [B]."""
    torch = _torch()
    lib = load()
    _need(target, "target")
    dev = target.device
    B, G1, V = target.shape
    G = G1 - 1
    _need(draft, "draft", dev, None, (B, G, V))
    _need(tokens, "tokens", dev, torch.int32, (B, G))
    _need(seeds, "seeds", dev, torch.int64, (B,))
    if out is None:
        out = dict(n=torch.empty((B,), dtype=torch.int32, device=dev),
                   committed=torch.empty((B, G1), dtype=torch.int32, device=dev),
                   bonus=torch.empty((B,), dtype=torch.int32, device=dev),
                   near=torch.empty((B,), dtype=torch.int32, device=dev))
    if ws is None:
        ws = workspace(OP_VERIFY_TOPK, B, G, V, 0, dev, stream)
    code = lib.spec_verify_topk(_ptr(target), _dtype_code(target), _ptr(draft), _dtype_code(draft), _ptr(tokens), B, G,
                                V, int(top_k), float(top_p), _ptr(seeds), _ptr(out["n"]), _ptr(out["committed"]),
                                _ptr(out["bonus"]), _ptr(out.get("near")), _ptr(ws), ws.numel(), _stream(stream))
    _check(code, "spec_verify_topk")
    out["ws"] = ws
    return out


def e2etv_shard(target, draft, n_branches, Wb, total_branches, ws=None, out=None, stream=None):
    """spec_e2etv_shard: one shard of a batch of ``total_branches`` branches.  target, draft
    bf16 [n_branches*Wb, V].  Returns a dict of device tensors: a, surv [R] float32,
    msum [1] float32 (this shard's part of the mean survival), grad bf16 [R, V]."""
    torch = _torch()
    lib = load()
    _need(target, "target", None, torch.bfloat16)
    dev = target.device
    R, V = target.shape
    if R != n_branches * Wb:
        raise ValueError("target must have n_branches * Wb rows")
    _need(draft, "draft", dev, torch.bfloat16, (R, V))
    if out is None:
        out = dict(
            a=torch.empty((R,), dtype=torch.float32, device=dev),
            surv=torch.empty((R,), dtype=torch.float32, device=dev),
            msum=torch.empty((1,), dtype=torch.float32, device=dev),
            grad=torch.empty((R, V), dtype=torch.bfloat16, device=dev),
        )
    if ws is None:
        ws = workspace(OP_E2ETV, n_branches, Wb, V, 0, dev, stream)
    code = lib.spec_e2etv_shard(_ptr(target), _ptr(draft), n_branches, Wb, V, int(total_branches), _ptr(out["a"]),
                                _ptr(out["surv"]), _ptr(out["msum"]), _ptr(out["grad"]), _ptr(ws), ws.numel(),
                                _stream(stream))
    _check(code, "spec_e2etv_shard")
    out["ws"] = ws
    return out


def e2etv(target, draft, n_branches, Wb, ws=None, out=None, stream=None):
    """spec_e2etv.  target, draft bf16 [n_branches*Wb, V] branch-major.  Returns a dict of
    device tensors: a, surv [R] float32, loss [1] float32, grad bf16 [R, V]."""
    torch = _torch()
    lib = load()
    _need(target, "target", None, torch.bfloat16)
    dev = target.device
    R, V = target.shape
    if R != n_branches * Wb:
        raise ValueError("target must have n_branches * Wb rows")
    _need(draft, "draft", dev, torch.bfloat16, (R, V))
    if out is None:
        out = dict(
            a=torch.empty((R,), dtype=torch.float32, device=dev),
            surv=torch.empty((R,), dtype=torch.float32, device=dev),
            loss=torch.empty((1,), dtype=torch.float32, device=dev),
            grad=torch.empty((R, V), dtype=torch.bfloat16, device=dev),
        )
    if ws is None:
        ws = workspace(OP_E2ETV, n_branches, Wb, V, 0, dev, stream)
    code = lib.spec_e2etv(_ptr(target), _ptr(draft), n_branches, Wb, V, _ptr(out["a"]), _ptr(out["surv"]),
                          _ptr(out["loss"]), _ptr(out["grad"]), _ptr(ws), ws.numel(), _stream(stream))
    _check(code, "spec_e2etv")
    out["ws"] = ws
    return out


def tree_select(parent, conf, m, out=None, stream=None):
    """spec_tree_select.  parent int32 [n_trees, n_nodes], conf float32 [n_trees, n_nodes].
    Returns a dict of device tensors: score float64 [n_trees, n_nodes], keep int32
    [n_trees, n_nodes] (1 = kept), selected int32 [n_trees, m] (ascending, then -1)."""
    torch = _torch()
    lib = load()
    _need(parent, "parent", None, torch.int32)
    if parent.dim() != 2:
        raise ValueError("parent must be [n_trees, n_nodes]")
    dev = parent.device
    T, n = parent.shape
    _need(conf, "conf", dev, torch.float32, (T, n))
    m = int(m)
    if out is None:
        out = dict(score=torch.empty((T, n), dtype=torch.float64, device=dev),
                   keep=torch.empty((T, n), dtype=torch.int32, device=dev),
                   selected=torch.empty((T, max(m, 0)), dtype=torch.int32, device=dev))
    code = lib.spec_tree_select(_ptr(parent), _ptr(conf), T, n, m, _ptr(out.get("score")), _ptr(out["keep"]),
                                _ptr(out.get("selected")) if m > 0 else _ptr(None), _stream(stream))
    _check(code, "spec_tree_select")
    return out


def tree_verify(target, parent, token, keep=None, ws=None, out=None, stream=None):
    """spec_tree_verify (T=0).  target f32/bf16 [n_trees, n_nodes + 1, V] (root row first);
    parent, token int32 [n_trees, n_nodes]; keep int32 [n_trees, n_nodes] or None (all).
    Returns a dict of device tensors: n [n_trees], path [n_trees, n_nodes], committed
    [n_trees, n_nodes + 1], bonus [n_trees]."""
    torch = _torch()
    lib = load()
    _need(target, "target")
    if target.dim() != 3:
        raise ValueError("target must be [n_trees, n_nodes + 1, V]")
    dev = target.device
    T, R, V = target.shape
    n = R - 1
    if n > 0:
        _need(parent, "parent", dev, torch.int32, (T, n))
        _need(token, "token", dev, torch.int32, (T, n))
        if keep is not None:
            _need(keep, "keep", dev, torch.int32, (T, n))
    if out is None:
        out = dict(n=torch.empty((T,), dtype=torch.int32, device=dev),
                   path=torch.empty((T, n), dtype=torch.int32, device=dev),
                   committed=torch.empty((T, R), dtype=torch.int32, device=dev),
                   bonus=torch.empty((T,), dtype=torch.int32, device=dev))
    if ws is None:
        ws = workspace(OP_TREE_VERIFY, T, n, V, 0, dev, stream)
    code = lib.spec_tree_verify(_ptr(target), _dtype_code(target), _ptr(parent if n > 0 else None),
                                _ptr(token if n > 0 else None), _ptr(keep if n > 0 else None), T, n, V,
                                _ptr(out["n"]), _ptr(out["path"]) if n > 0 else _ptr(None), _ptr(out["committed"]),
                                _ptr(out["bonus"]), _ptr(ws), ws.numel(), _stream(stream))
    _check(code, "spec_tree_verify")
    out["ws"] = ws
    return out


def draft_block_topk(logits, anchor, U, Wt, top_k, top_p, seeds, ws=None, out=None, stream=None):
    """spec_draft_block_topk (T=1, filtered draws).  logits [B, gamma, V] f32/bf16; anchor
    [B] int32; U, Wt bf16 [V, r] or None; seeds [B] int64.  Returns a dict of device
    tensors: tokens [B, gamma] int32, conf and qtok [B, gamma] float32."""
    torch = _torch()
    lib = load()
    _need(logits, "logits")
    dev = logits.device
    B, G, V = logits.shape
    _need(anchor, "anchor", dev, torch.int32, (B,))
    _need(seeds, "seeds", dev, torch.int64, (B,))
    r = 0
    if U is not None:
        r = U.shape[1]
        _need(U, "U", dev, torch.bfloat16, (V, r))
        _need(Wt, "Wt", dev, torch.bfloat16, (V, r))
    if out is None:
        out = dict(tokens=torch.empty((B, G), dtype=torch.int32, device=dev),
                   conf=torch.empty((B, G), dtype=torch.float32, device=dev),
                   qtok=torch.empty((B, G), dtype=torch.float32, device=dev))
    if ws is None:
        ws = workspace(OP_DRAFT_TOPK, B, G, V, r, dev, stream)
    code = lib.spec_draft_block_topk(_ptr(logits), _dtype_code(logits), _ptr(anchor), _ptr(U), _ptr(Wt), BF16, r, B, G,
                                     V, int(top_k), float(top_p), _ptr(seeds), _ptr(out["tokens"]), _ptr(out["conf"]),
                                     _ptr(out.get("qtok")), _ptr(ws), ws.numel(), _stream(stream))
    _check(code, "spec_draft_block_topk")
    out["ws"] = ws
    return out


# ---------------------------------------------------------------------------------
# the rows before verification, and what a drafter learns from them
# ---------------------------------------------------------------------------------
_PROCESS_NAMES = ("history", "lengths", "prompt_lengths", "block", "repetition", "frequency", "presence",
                  "temperature", "bias_ids", "bias_values", "mask")


def process_logits(logits, history=None, lengths=None, prompt_lengths=None, block=None, repetition=None,
                   frequency=None, presence=None, bias_ids=None, bias_values=None, mask=None, temperature=None,
                   ws=None, out=None, stream=None):
    """spec_process_logits.  logits [B, R, V] f32/bf16 (rows may lie further apart than V);
    history int32 [B, Lmax], lengths and prompt_lengths int32 [B]; block int32 [B, R - 1],
    the block's tokens; repetition, frequency, presence, temperature float32 [B]; bias_ids
    int32 and bias_values float32 [B, n]; mask int32 [B, R, ceil(V / 32)] or, shared by a
    request's rows, [B, ceil(V / 32)], a set bit for an allowed token.  Every one of them
    but logits may be None.  ``out=dict(logits=...)`` may be logits itself.  Returns a dict
    of device tensors: logits."""
    torch = _torch()
    lib = _lib or load()
    ld = _need_rows(logits, "logits")
    if logits.dim() != 3:
        raise ValueError("logits must be [B, R, V]")
    dev, i32, f32 = logits.device, torch.int32, torch.float32
    if _away(dev, stream):
        with torch.cuda.device(dev):
            return process_logits(logits, history, lengths, prompt_lengths, block, repetition, frequency, presence,
                                  bias_ids, bias_values, mask, temperature, ws, out, stream)
    B, R, V = logits.shape
    Lmax = nb = 0
    if history is not None:
        if history.dim() != 2:
            raise ValueError(f"history must be [{B}, Lmax], got {tuple(history.shape)}")
        Lmax = history.shape[1]
    if (bias_ids is None) != (bias_values is None):
        raise ValueError("bias_ids and bias_values go together")
    if bias_ids is not None:
        if bias_ids.dim() != 2:
            raise ValueError(f"bias_ids must be [{B}, n], got {tuple(bias_ids.shape)}")
        nb = bias_ids.shape[1]
    _need_ints("process_logits", B, R, V, ld, Lmax, nb)
    W = (V + 31) // 32
    mask_rows, masks = (R, (B, R, W)) if mask is not None and mask.dim() == 3 else (1, (B, W))
    per, biases = (B,), (B, nb)
    (a_hist, a_len, a_prompt, a_block, a_rep, a_freq, a_pres, a_temp, a_ids, a_values, a_mask) = _addrs(
        dev, _PROCESS_NAMES,
        (history, lengths, prompt_lengths, block, repetition, frequency, presence, temperature, bias_ids,
         bias_values, mask),
        (i32, i32, i32, i32, f32, f32, f32, f32, i32, f32, i32),
        ((B, Lmax), per, per, (B, R - 1), per, per, per, per, biases, biases, masks))
    if out is None:
        with _made_on(stream):
            out = dict(logits=_rows_like(logits, ld))
    else:
        _need_same_rows(out.get("logits"), "out's logits", logits, ld)
    if ws is None:
        with _made_on(stream):
            ws = workspace(OP_PROCESS_LOGITS, B, R, V, 0, dev, stream)
    code = lib.spec_process_logits(
        logits.data_ptr(), _dtype_code(logits), B, R, V, ld, a_hist if Lmax else None, Lmax, a_len, a_prompt,
        a_block if R > 1 else None, a_rep, a_freq, a_pres, a_temp, a_ids if nb else None, a_values if nb else None,
        nb, a_mask, mask_rows, out["logits"].data_ptr(), ws.data_ptr(), _ws_bytes(ws, dev), _stream(stream))
    if code != OK:
        raise SpecError(code, "spec_process_logits")
    out["ws"] = ws
    return out


def top_logits(logits, k, temperature=1.0, ws=None, out=None, stream=None):
    """spec_top_logits.  logits [..., V] f32/bf16 (rows may lie further apart than V).
    Returns a dict of device tensors: values float32 and ids int32 [..., k], tail and lse
    float32 [...]."""
    torch = _torch()
    lib = _lib or load()
    ld = _need_rows(logits, "logits")
    dev, shape, k = logits.device, logits.shape, int(k)
    if _away(dev, stream):
        with torch.cuda.device(dev):
            return top_logits(logits, k, temperature, ws, out, stream)
    lead, V = shape[:-1], shape[-1]
    rows = logits.numel() // V if V else 0
    _need_ints("top_logits", rows, V, ld, k)
    if out is None:
        with _made_on(stream):
            sized = (*lead, max(k, 0))
            out = dict(values=torch.empty(sized, dtype=torch.float32, device=dev),
                       ids=torch.empty(sized, dtype=torch.int32, device=dev),
                       tail=torch.empty(lead, dtype=torch.float32, device=dev),
                       lse=torch.empty(lead, dtype=torch.float32, device=dev))
    else:
        _need_out(out, dev, values=(torch.float32, (*lead, k)), ids=(torch.int32, (*lead, k)),
                  tail=(torch.float32, lead), lse=(torch.float32, lead))
    if ws is None:
        with _made_on(stream):
            ws = workspace(OP_TOP_LOGITS, rows, k, V, 0, dev, stream)
    lse = out.get("lse")
    code = lib.spec_top_logits(logits.data_ptr(), _dtype_code(logits), rows, V, ld, k, float(temperature),
                               out["values"].data_ptr(), out["ids"].data_ptr(), out["tail"].data_ptr(),
                               None if lse is None else lse.data_ptr(), ws.data_ptr(), _ws_bytes(ws, dev),
                               _stream(stream))
    if code != OK:
        raise SpecError(code, "spec_top_logits")
    out["ws"] = ws
    return out


def distill(student, values, ids, tail=None, weight=None, temperature=1.0, grad=False, ws=None, out=None,
            stream=None):
    """spec_distill.  student [..., V] f32/bf16 (rows may lie further apart than V); values
    f32/bf16 and ids int32 [..., K]; tail and weight float32 [...] or None.  Returns a dict
    of device tensors: loss and lse float32 [...] and, with ``grad``, grad of the student's
    type and layout (``out["grad"]`` may be student itself)."""
    torch = _torch()
    lib = _lib or load()
    ld = _need_rows(student, "student")
    dev, shape = student.device, student.shape
    if _away(dev, stream):
        with torch.cuda.device(dev):
            return distill(student, values, ids, tail, weight, temperature, grad, ws, out, stream)
    lead, V = shape[:-1], shape[-1]
    rows = student.numel() // V if V else 0
    K = ids.shape[-1] if ids is not None and ids.dim() else 0
    _need_ints("distill", rows, V, ld, K)
    if ids is None or values is None:
        raise ValueError("values and ids are required")
    named = (*lead, K)
    a_values, a_ids, a_tail, a_weight = _addrs(
        dev, ("values", "ids", "tail", "weight"), (values, ids, tail, weight),
        (values.dtype, torch.int32, torch.float32, torch.float32), (named, named, lead, lead))
    if out is None:
        with _made_on(stream):
            out = dict(loss=torch.empty(lead, dtype=torch.float32, device=dev),
                       lse=torch.empty(lead, dtype=torch.float32, device=dev))
            if grad:
                out["grad"] = _rows_like(student, ld)
    else:
        _need_out(out, dev, loss=(torch.float32, lead), lse=(torch.float32, lead))
        if grad:
            _need_same_rows(out.get("grad"), "grad", student, ld)
    if ws is None:
        with _made_on(stream):
            ws = workspace(OP_DISTILL, rows, K, V, 0, dev, stream)
    lse = out.get("lse")
    code = lib.spec_distill(student.data_ptr(), _dtype_code(student), rows, V, ld, a_values, _dtype_code(values),
                            a_ids, K, a_tail, a_weight, float(temperature), out["loss"].data_ptr(),
                            None if lse is None else lse.data_ptr(), out["grad"].data_ptr() if grad else None,
                            ws.data_ptr(), _ws_bytes(ws, dev), _stream(stream))
    if code != OK:
        raise SpecError(code, "spec_distill")
    out["ws"] = ws
    return out


# ---------------------------------------------------------------------------------
# a drafter's training step
# ---------------------------------------------------------------------------------
def policy_loss(logits, tokens, old_logp, advantage, ref_logp=None, weight=None, temperature=1.0, clip=(0.2, 0.2),
                kl=0.0, grad=False, ws=None, out=None, stream=None):
    """spec_policy_loss.  logits [..., V] f32/bf16 (rows may lie further apart than V); tokens
    int32 [...]; old_logp, advantage, ref_logp (needed where kl > 0) and weight (or None) float32
    [...]; clip the ratio's room below and above 1.  Returns a dict of device tensors: loss and
    logp float32 [...] and, with ``grad``, grad of the logits' type and layout (``out["grad"]``
    may be logits itself)."""
    torch = _torch()
    lib = _lib or load()
    ld = _need_rows(logits, "logits")
    dev, shape = logits.device, logits.shape
    if _away(dev, stream):
        with torch.cuda.device(dev):
            return policy_loss(logits, tokens, old_logp, advantage, ref_logp, weight, temperature, clip, kl, grad, ws,
                               out, stream)
    lead, V = shape[:-1], shape[-1]
    rows = logits.numel() // V if V else 0
    _need_ints("policy_loss", rows, V, ld)
    if tokens is None or old_logp is None or advantage is None:
        raise ValueError("tokens, old_logp and advantage are required")
    if kl > 0 and ref_logp is None:
        raise ValueError("ref_logp is required where kl > 0")
    low, high = clip
    f32 = torch.float32
    a_tok, a_old, a_adv, a_ref, a_weight = _addrs(
        dev, ("tokens", "old_logp", "advantage", "ref_logp", "weight"), (tokens, old_logp, advantage, ref_logp, weight),
        (torch.int32, f32, f32, f32, f32), (lead,) * 5)
    if out is None:
        with _made_on(stream):
            out = dict(loss=torch.empty_like(old_logp), logp=torch.empty_like(old_logp))   # float32 [...], as checked
            if grad:
                out["grad"] = _rows_like(logits, ld)
    else:
        _need_out(out, dev, loss=(f32, lead), logp=(f32, lead))
        if grad:
            _need_same_rows(out.get("grad"), "grad", logits, ld)
    if ws is None:
        with _made_on(stream):
            ws = workspace(OP_POLICY_LOSS, rows, 1, V, 0, dev, stream)
    code = lib.spec_policy_loss(
        logits.data_ptr(), _dtype_code(logits), rows, V, ld, a_tok, a_old, a_adv, a_ref, a_weight, float(temperature),
        float(low), float(high), float(kl), out["loss"].data_ptr(), out["logp"].data_ptr(),
        out["grad"].data_ptr() if grad else None, ws.data_ptr(), _ws_bytes(ws, dev), _stream(stream))
    if code != OK:
        raise SpecError(code, "spec_policy_loss")
    out["ws"] = ws
    return out


def markov_grad(grad, anchor, tokens, U, Wt, dtype=None, ws=None, out=None, stream=None):
    """spec_markov_grad.  grad [B, gamma, V] f32/bf16, the biased rows' gradient (rows may lie
    further apart than V); anchor int32 [B] and tokens int32 [B, gamma] as draft_block takes and
    gives them (-1: the rows behind count for nothing; tokens may be None where gamma is 1);
    U, Wt [V, r] f32/bf16; ``dtype`` the outputs' type, the weights' by default.  Returns a dict
    of device tensors: U and Wt [V, r], their gradients."""
    torch = _torch()
    lib = _lib or load()
    ld = _need_rows(grad, "grad")
    if grad.dim() != 3:
        raise ValueError("grad must be [B, gamma, V]")
    dev = grad.device
    if _away(dev, stream):
        with torch.cuda.device(dev):
            return markov_grad(grad, anchor, tokens, U, Wt, dtype, ws, out, stream)
    B, gamma, V = grad.shape
    if U is None or Wt is None or anchor is None or (tokens is None and gamma != 1):
        raise ValueError("anchor, tokens, U and Wt are required")
    if U.dim() != 2 or U.shape[0] != V:
        raise ValueError(f"U must be [{V}, r], got {tuple(U.shape)}")
    r = U.shape[1]
    _need_ints("markov_grad", B, gamma, V, ld, r)
    wdt = _dtype_code(U)
    a_anchor, a_tokens, a_U, a_Wt = _addrs(dev, ("anchor", "tokens", "U", "Wt"), (anchor, tokens, U, Wt),
                                           (torch.int32, torch.int32, U.dtype, U.dtype),
                                           ((B,), (B, gamma), U.shape, U.shape))
    if out is None:
        with _made_on(stream):
            out = dict(U=torch.empty_like(U, dtype=dtype), Wt=torch.empty_like(U, dtype=dtype))
    else:
        dtype = dtype or (U.dtype if out.get("U") is None else out["U"].dtype)
        _need_out(out, dev, U=(dtype, (V, r)), Wt=(dtype, (V, r)))
    odt = _dtype_code(out["U"])
    if ws is None:
        with _made_on(stream):
            ws = workspace(OP_MARKOV_GRAD, B, gamma, V, r, dev, stream)
    code = lib.spec_markov_grad(
        grad.data_ptr(), _dtype_code(grad), B, gamma, V, ld, a_anchor, a_tokens, a_U, a_Wt, wdt, r,
        out["U"].data_ptr(), out["Wt"].data_ptr(), odt, ws.data_ptr(), _ws_bytes(ws, dev), _stream(stream))
    if code != OK:
        raise SpecError(code, "spec_markov_grad")
    out["ws"] = ws
    return out


def adamw_state(param, bits=32, master=None):
    """A parameter's state for adamw: a dict of device tensors, m and v (zeros), in 8 bits also
    m_scale and v_scale, for a bf16 parameter its float32 master (the parameter's values, or
    the tensor given).  Over many steps v in 8 bits settles 3 to 6 % above v in 32, and its root
    scatters by some 15 % (spec_adamw says why)."""
    torch = _torch()
    dev, shape = param.device, param.shape
    if bits == 32:
        s = {k: torch.zeros(shape, dtype=torch.float32, device=dev) for k in ("m", "v")}
    elif bits == 8:
        blocks = (param.numel() + ADAMW_BLOCK - 1) // ADAMW_BLOCK
        s = {k: torch.zeros(shape, dtype=torch.float8_e4m3fn, device=dev) for k in ("m", "v")}
        s.update({k: torch.zeros((blocks,), dtype=torch.float32, device=dev) for k in ("m_scale", "v_scale")})
    else:
        raise ValueError(f"a state has 32 or 8 bits, got {bits}")
    if _dtype_code(param) == BF16:
        s["master"] = param.detach().float() if master is None else master
    elif master is not None:
        raise ValueError("a float32 parameter has no master")
    return s


class AdamwTable:
    """What adamw steps over: the tensors of adamw_table, and their addresses for the library."""

    def __init__(self, params, grads, states, device, entries):
        self.params, self.grads, self.states, self.device, self.entries = params, grads, states, device, entries
        # the memory that the addresses are of, whatever a tensor is given later (p.data = ...)
        self.storages = [t.untyped_storage() for p, g, s in zip(params, grads, states)
                         for t in (p, g, *map(s.get, _STATE)) if t is not None]
        # what autograd may hold for a backward pass
        self.tracked = [p for p in params if p.requires_grad]
        # parameters whose gradient is the one that a backward pass adds to
        self.leaves = [(i, p, g) for i, (p, g) in enumerate(zip(params, grads))
                       if p.requires_grad and p.is_leaf and p.grad is g]

    def __len__(self):
        return len(self.params)


def _distinct(spans):
    """Refuses memory that a step writes and uses a second time (one parameter listed twice, tied
    weights): spans are (address, bytes, written, name)."""
    last = last_written = (0, None)     # where what lies furthest ends: of all so far, of the written ones
    for at, size, written, name in sorted((s for s in spans if s[1] > 0), key=lambda s: s[0]):
        end, other = last if written else last_written
        if at < end:
            raise ValueError(f"{name} overlaps {other}")
        last = max(last, (at + size, name), key=lambda x: x[0])
        if written:
            last_written = max(last_written, (at + size, name), key=lambda x: x[0])


def adamw_table(params, grads, states):
    """The tensors of an AdamW step, checked once and kept: lists of parameters (f32/bf16), of
    their gradients (f32/bf16, read anew at every step) and of their states (adamw_state's dicts;
    32 and 8 bits may be mixed).  Steps write the parameters and states in place, so none of them may
    overlap another tensor of the table; a tensor that is given other memory later needs a new table.
    So does a parameter whose .grad becomes other memory: zero_grad has to keep it (set_to_none=False); a
    step over a table made of p.grad refuses one that is not there any more."""
    torch = _torch()
    params, grads, states = list(params), list(grads), list(states)
    if not len(params) == len(grads) == len(states):
        raise ValueError(f"{len(params)} parameters, {len(grads)} gradients and {len(states)} states")
    if not params:
        raise ValueError("an empty table")
    if len(params) > 65536:
        raise SpecError(2, f"adamw_table({len(params)} tensors)")
    dev = params[0].device
    f32, f8 = torch.float32, torch.float8_e4m3fn
    entries = (AdamwTensor * len(params))()
    spans = []
    for i, (p, g, s, e) in enumerate(zip(params, grads, states, entries)):
        _need(p, f"parameter {i}", dev)
        e.param_dtype = _dtype_code(p)
        _need(g, f"gradient {i}", dev, None, p.shape)
        e.grad_dtype = _dtype_code(g)
        for k in ("m", "v"):
            if s.get(k) is None:
                raise ValueError(f"state {i} has no {k}")
        packed = s["m"].dtype == f8
        for k in ("m", "v"):
            _need(s[k], f"state {i}'s {k}", dev, f8 if packed else f32, p.shape)
            if packed:
                _need(s.get(k + "_scale"), f"state {i}'s {k}_scale", dev, f32,
                      ((p.numel() + ADAMW_BLOCK - 1) // ADAMW_BLOCK,))
        if e.param_dtype == BF16:
            _need(s.get("master"), f"state {i}'s master", dev, f32, p.shape)
            e.master = s["master"].data_ptr()
        elif s.get("master") is not None:
            raise ValueError(f"state {i}: a float32 parameter has no master")
        e.param, e.grad, e.m, e.v, e.n = p.data_ptr(), g.data_ptr(), s["m"].data_ptr(), s["v"].data_ptr(), p.numel()
        e.state_bits = 8 if packed else 32
        if packed:
            e.m_scale, e.v_scale = s["m_scale"].data_ptr(), s["v_scale"].data_ptr()
        used = [("parameter", p), ("gradient", g)] + [(f"{k} of state", s.get(k)) for k in _STATE]
        spans += [(t.data_ptr(), t.numel() * t.element_size(), name != "gradient", f"{name} {i}")
                  for name, t in used if t is not None]
    _distinct(spans)
    return AdamwTable(params, grads, states, dev, entries)


def adamw(table, step, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, grad_scale=None, seed=0, ws=None,
          stream=None):
    """spec_adamw: one AdamW step over an adamw_table, in place.  step int32 [1] on the device,
    the steps taken so far, which the call counts up; grad_scale float32 [1] on the device or None,
    a factor of all gradients; seed the 8-bit states' random rounding.  lr and weight_decay are the whole
    table's (parameters with others need a table and a step of their own) and stay what they are in a
    captured call.  A backward pass through parameters as they were before the step is refused by
    torch, but not after a replayed graph, which raises no versions.  Returns a dict: step."""
    torch = _torch()
    lib = _lib or load()
    dev = table.device
    if _away(dev, stream):
        with torch.cuda.device(dev):
            return adamw(table, step, lr, betas, eps, weight_decay, grad_scale, seed, ws, stream)
    a_step, a_scale = _addrs(dev, ("step", "grad_scale"), (step, grad_scale), (torch.int32, torch.float32), ((1,), (1,)))
    if a_step is None:
        raise ValueError("step is required")
    for i, p, g in table.leaves:
        if p.grad is not g and (p.grad is None or p.grad.data_ptr() != g.data_ptr()):
            raise ValueError(f"parameter {i}'s gradient is not the table's any more (zero_grad(set_to_none=True)?)")
    if ws is None:
        with _made_on(stream):
            ws = workspace(OP_ADAMW, len(table), 1, 1, 0, dev, stream)
    code = lib.spec_adamw(table.entries, len(table), a_step, float(lr), float(betas[0]), float(betas[1]), float(eps),
                          float(weight_decay), a_scale, int(seed) & 0xFFFFFFFFFFFFFFFF, ws.data_ptr(),
                          _ws_bytes(ws, dev), _stream(stream))
    if code != OK:
        raise SpecError(code, "spec_adamw")
    if table.tracked:   # so that a backward pass through what they were before is refused
        torch.autograd.graph.increment_version(table.tracked)
    return dict(step=step, ws=ws)
