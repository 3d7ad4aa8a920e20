"""Python binding of the draft-tree C ABI (include/dtree.h).

Argument marshalling only: every step of build, mask and verify runs in the
CUDA kernels of libdtree.so.  Tensors must be CUDA tensors, contiguous, of the
documented dtype; the library writes into caller-owned buffers on the current
torch stream (or the stream given).  A missing or unloadable library raises --
there is no other code path.
"""
import contextlib
import ctypes
import dataclasses
import math
import os

import torch

from . import build as _build

DT_MODE = {"ddtree": 0, "dartree": 1, "talon": 2, "heap": 3}
BUDGET_POLICY = {"topb": 0, "uniform": 1}
DT_BF16, DT_F32 = 0, 1
DT_DEV_BAD_TREE, DT_DEV_TIMEOUT, DT_DEV_BESTFIRST, DT_DEV_BAD_CACHE = 0x1, 0x2, 0x4, 0x8
DT_DEV_VIOLATION_SHIFT = 8
DT_STAGE1_CLUSTER, DT_STAGE1_ROWS = 1, 2
# acceptance rules of dt_verify_rule
VERIFY_RULES = {"greedy": 0, "ratio": 1, "iter_residual": 2, "target_match": 3}
MAX_NODES = 1025
MAX_KC = 1024
MAX_TOP = 32
PAGE_SIZES = (16, 32, 64, 128)

_i32 = ctypes.c_int32
_i64 = ctypes.c_int64
_vp = ctypes.c_void_p


class TdesStruct(ctypes.Structure):
    _fields_ = [("H", _i32), ("Ap", _vp), ("Ac", _vp), ("Dd", _vp), ("w", _vp), ("b0", ctypes.c_float),
                ("s", ctypes.c_float)]


class BuildParams(ctypes.Structure):
    _fields_ = [("mode", _i32), ("batch", _i32), ("L", _i32), ("V", _i32), ("dtype", _i32),
                ("K", _i32), ("B", _i32), ("W", _i32), ("beta", ctypes.c_float), ("R", _i32),
                ("U", _vp), ("Vt", _vp), ("root_tok", _vp), ("talon_k", _i32),
                ("log_mu", ctypes.c_float), ("N", _i32), ("markov_norm", _i32),
                ("tdes", ctypes.POINTER(TdesStruct)), ("budget_policy", _i32), ("budget", _vp)]


class SabaStruct(ctypes.Structure):
    _fields_ = [("window", _i32), ("c_verify", ctypes.c_float), ("c_fixed", ctypes.c_float), ("B_min", _i32),
                ("B_max", _i32)]


class TreeStruct(ctypes.Structure):
    _fields_ = [("max_nodes", _i32), ("Kc", _i32), ("L", _i32), ("node_tok", _vp), ("parent", _vp),
                ("depth", _vp), ("rank", _vp), ("score", _vp), ("n_nodes", _vp), ("lse", _vp),
                ("cand_id", _vp), ("cand_lp", _vp), ("status", _vp)]


class CacheStruct(ctypes.Structure):
    _fields_ = [("n_pages", _i32), ("page", _i32), ("Hkv", _i32), ("D", _i32), ("max_pages", _i32), ("k", _vp),
                ("v", _vp), ("k_scale", _vp), ("v_scale", _vp), ("table", _vp), ("len", _vp)]


class RopeStruct(ctypes.Structure):
    _fields_ = [("cos", _vp), ("sin", _vp), ("max_pos", _i32), ("rot", _i32), ("interleaved", _i32)]


class RowsStruct(ctypes.Structure):
    _fields_ = [("ptr", _vp), ("stride_b", _i64), ("stride_n", _i64), ("stride_h", _i64)]


_LIB = None


def lib():
    """Load libdtree.so (compiling it first if it has never been built)."""
    global _LIB
    if _LIB is None:
        path = _build.LIB
        if not os.path.exists(path):
            path = _build.build()
        L = ctypes.CDLL(path)
        bp = ctypes.POINTER(BuildParams)
        tp = ctypes.POINTER(TreeStruct)
        L.dt_workspace_size.restype = ctypes.c_size_t
        L.dt_workspace_size.argtypes = [bp, ctypes.POINTER(ctypes.c_int)]
        L.dt_candidates.restype = _i32
        L.dt_candidates.argtypes = [bp, _vp, tp, _vp]
        L.dt_markov_norm.restype = _i32
        L.dt_markov_norm.argtypes = [bp, _vp, tp, _vp, ctypes.c_size_t, _vp]
        L.dt_stage1_plan.restype = _i32
        L.dt_stage1_plan.argtypes = [bp, ctypes.POINTER(_i32), ctypes.POINTER(_i32)]
        L.dt_stage1_ceiling.restype = _i32
        L.dt_stage1_ceiling.argtypes = [bp, _vp, _vp, _vp, _vp]
        L.dt_select.restype = _i32
        L.dt_select.argtypes = [bp, tp, _vp, ctypes.c_size_t, _vp]
        L.dt_build_tree.restype = _i32
        L.dt_build_tree.argtypes = [bp, _vp, tp, _vp, ctypes.c_size_t, _vp]
        L.dt_tree_mask.restype = _i32
        L.dt_tree_mask.argtypes = [tp, _i32, _i32, _vp, _vp, _vp]
        L.dt_verify.restype = _i32
        L.dt_saba_budget.restype = _i32
        L.dt_saba_budget.argtypes = [ctypes.POINTER(SabaStruct), tp, _i32, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp]
        L.dt_verify_markov.restype = _i32
        L.dt_verify_markov.argtypes = [bp, tp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
        L.dt_verify_rule.restype = _i32
        L.dt_verify_rule.argtypes = [tp, _i32, _i32, _i32, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp]
        L.dt_verify.argtypes = [tp, _i32, _i32, _i32, _vp, _vp, _vp, ctypes.c_float, _vp, _vp, _vp, _vp, _vp,
                                _vp]
        L.dt_select_dartree_noalloc.restype = _i32
        L.dt_select_dartree_noalloc.argtypes = [bp, tp, _vp]
        L.dt_test_wait_fault.restype = _i32
        L.dt_test_wait_fault.argtypes = [_i32, ctypes.c_int64]
        cp, rp, xp = ctypes.POINTER(CacheStruct), ctypes.POINTER(RopeStruct), ctypes.POINTER(RowsStruct)
        L.dt_kv_append.restype = _i32
        L.dt_kv_append.argtypes = [cp, rp, _i32, _i32, _i32, xp, xp, _vp, _i32, _vp, _i32, _vp, _vp, _vp]
        L.dt_tree_attention_workspace.restype = ctypes.c_size_t
        L.dt_tree_attention_workspace.argtypes = [cp, _i32, _i32, _i32]
        L.dt_tree_attention.restype = _i32
        L.dt_tree_attention.argtypes = [cp, rp, _i32, _i32, _i32, xp, xp, xp, _vp, _vp, _vp, ctypes.c_float, _vp, _vp,
                                        ctypes.c_size_t, _vp, _vp]
        # a 4-bit cache has the same fields, k_scale and v_scale pointing to bytes
        L.dt_kv_append4.restype = L.dt_tree_attention4.restype = _i32
        L.dt_kv_append4.argtypes = L.dt_kv_append.argtypes
        L.dt_tree_attention4.argtypes = L.dt_tree_attention.argtypes
        L.dt_tree_attention4_workspace.restype = ctypes.c_size_t
        L.dt_tree_attention4_workspace.argtypes = L.dt_tree_attention_workspace.argtypes
        L.dt_kv_read.restype = L.dt_kv_read4.restype = _i32
        L.dt_kv_read.argtypes = L.dt_kv_read4.argtypes = [cp, _i32, _vp, _i32, _vp, _vp, _i32, _i32, xp, xp, _vp, _vp]
        L.dt_qk_norm.restype = _i32
        L.dt_qk_norm.argtypes = [_i32, _i32, _i32, _i32, _i32, _i32, xp, xp, _vp, _i32, _vp, _i32, ctypes.c_float, rp,
                                 _vp, _vp, _vp, xp, xp, _vp, _vp]
        L.dt_token_logprobs.restype = _i32
        L.dt_token_logprobs.argtypes = [_vp, _i32, _i32, _i32, _i32, _i64, _i64, _vp, _vp, _i32, _i32, _vp, _vp,
                                        _vp, _vp, _vp, _vp]
        L.dt_status_str.restype = ctypes.c_char_p
        L.dt_status_str.argtypes = [_i32]
        L.dt_version.restype = _i32
        _LIB = L
    return _LIB


PROBE = {"stage1": 0x1, "walk": 0x2, "normaliser": 0x4, "attention": 0x10}


def set_test_wait_fault(kernels=(), budget_cycles=2_000_000):
    """dt_test_wait_fault: make the named kernels' bounded waits run out once per
    staging step (a test of the timeout path); kernels=() turns it off."""
    mask = 0
    for k in kernels:
        mask |= PROBE[k]
    _check(lib().dt_test_wait_fault(mask, int(budget_cycles) if mask else 0), "dt_test_wait_fault")


class DtError(RuntimeError):
    pass


def _check(rc, what):
    if rc != 0:
        raise DtError("%s: %s (%d)" % (what, lib().dt_status_str(rc).decode(), rc))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    # the current stream's handle, without a Stream object (4 us of host time per call)
    return ctypes.c_void_p(_raw_stream(torch.cuda.current_device()))


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # None: torch without CUDA, which has no streams


def _on(stream):
    """Context in which a call allocates what its caller did not bring: on the stream that the call
    runs on, so that fills come before it and freed memory is not handed out while it runs."""
    return torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext()


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return DT_BF16
    if t.dtype == torch.float32:
        return DT_F32
    raise TypeError("logits must be bfloat16 or float32, got %s" % t.dtype)


def _need(t, dtype=None, name="tensor", numel=None):
    """A contiguous CUDA tensor (of dtype), holding at least numel elements: the
    C ABI takes bare pointers, so sizes are checked here, before any launch."""
    if t.is_cuda and t.is_contiguous() and (dtype is None or t.dtype == dtype) and (numel is None or t.numel() >= numel):
        return t
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    _need_numel(t, numel, name)
    return t


def _need_numel(t, numel, name):
    if numel is not None and t.numel() < numel:
        raise ValueError("%s holds %d elements, the call reads or writes %d" % (name, t.numel(), numel))


def _need_batch(tree, batch):
    """The tree buffers (dt_tree carries no batch size) must hold `batch` requests."""
    if batch > tree.batch:
        raise ValueError("the tree buffers hold %d requests, the call covers %d" % (tree.batch, batch))


def _need_logits(t, p, name="draft_logits"):
    """[batch, L, V] drafter logits of Params p's dtype."""
    _need(t, name=name, numel=p.batch * p.L * p.V)
    if _dtype_code(t) != (DT_BF16 if p.dtype == "bf16" else DT_F32):
        raise TypeError("%s must be %s for dtype=%r, got %s" % (name, "bfloat16" if p.dtype == "bf16" else "float32",
                                                                p.dtype, t.dtype))
    if t.shape[-1] != p.V:
        raise ValueError("%s rows must hold V = %d logits, got %d" % (name, p.V, t.shape[-1]))


def _need_workspace(workspace):
    ws, n = (workspace if workspace is not None else (None, 0))
    if ws is not None:
        _need(ws, name="workspace")
        if ws.numel() * ws.element_size() < n:
            raise ValueError("workspace holds %d bytes, %d were declared" % (ws.numel() * ws.element_size(), n))
    return ws, n


@dataclasses.dataclass
class Params:
    """Build parameters; mirrors dt_build_params."""
    mode: str
    batch: int
    L: int
    V: int
    dtype: str = "bf16"
    K: int = 0
    B: int = 0
    W: int = 0
    beta: float = 0.0
    R: int = 0
    U: torch.Tensor = None
    Vt: torch.Tensor = None
    root_tok: torch.Tensor = None
    talon_k: int = 0
    mu: float = 0.0
    N: int = 0
    markov_norm: bool = False  # DARTree: full-vocabulary normalised correction
    tdes: "Tdes" = None        # heap mode: TDES edge scorer
    budget_policy: str = "topb"  # DARTree: "uniform" = DARTree (fixed), per-depth widths from B
    budgets: torch.Tensor = None  # DDTree / heap: [batch] int32 per-request budgets (dt_build_params.budget)

    @property
    def Kc(self):
        return min(self.N, self.V) if self.mode == "talon" else self.K

    @property
    def budget(self):
        return self.N if self.mode == "talon" else self.B

    def struct(self, for_launch=True):
        """The dt_build_params block.  for_launch: check the device tensors it points
        to (the host-only queries, workspace_size and stage1_plan, read no tensor)."""
        log_mu = 0.0
        if self.mode == "talon":
            log_mu = float(torch.tensor(math.log(self.mu), dtype=torch.float64).float())
        bp = BuildParams(DT_MODE[self.mode], self.batch, self.L, self.V,
                         DT_BF16 if self.dtype == "bf16" else DT_F32, self.K, self.B, self.W,
                         self.beta, self.R if self.U is not None else 0, _ptr(self.U), _ptr(self.Vt),
                         _ptr(self.root_tok), self.talon_k, log_mu, self.N, int(bool(self.markov_norm)))
        if for_launch:
            if self.U is not None:
                _need(self.U, torch.float32, "U", numel=self.V * self.R)
                _need(self.Vt, torch.float32, "Vt", numel=self.V * self.R)
            if self.root_tok is not None:
                _need(self.root_tok, torch.int32, "root_tok", numel=self.batch)
            if self.budgets is not None:
                _need(self.budgets, torch.int32, "budgets", numel=self.batch)
        if self.tdes is not None:
            if for_launch:
                H = int(self.tdes.w.shape[0])
                _need_numel(self.tdes.Ap, self.V * H, "Ap")
                _need_numel(self.tdes.Ac, self.V * H, "Ac")
                _need_numel(self.tdes.Dd, self.L * H, "Dd")
            bp._tdes = self.tdes.struct()  # kept alive with the parameter block
            bp.tdes = ctypes.pointer(bp._tdes)
        bp.budget_policy = BUDGET_POLICY[self.budget_policy]
        if self.budgets is not None:
            bp.budget = _ptr(self.budgets)
        return bp


@dataclasses.dataclass
class Tdes:
    """TDES edge scorer (dt_tdes): per-token first-layer rows Ap, Ac [V, H], depth rows
    Dd [L, H] (bias included), output weights w [H], bias b0, scale s; fp32 device tensors."""
    Ap: torch.Tensor
    Ac: torch.Tensor
    Dd: torch.Tensor
    w: torch.Tensor
    b0: float = 0.0
    s: float = 1.0

    def struct(self):
        for name in ("Ap", "Ac", "Dd", "w"):
            _need(getattr(self, name), torch.float32, name)
        return TdesStruct(int(self.w.shape[0]), _ptr(self.Ap), _ptr(self.Ac), _ptr(self.Dd), _ptr(self.w),
                          float(self.b0), float(self.s))


class TreeBuffers:
    """Device buffers of a batch of trees (dt_tree)."""

    def __init__(self, batch, L, Kc, max_nodes, device="cuda"):
        i32 = dict(dtype=torch.int32, device=device)
        f32 = dict(dtype=torch.float32, device=device)
        self.batch, self.L, self.Kc, self.max_nodes = batch, L, Kc, max_nodes
        self.node_tok = torch.full((batch, max_nodes), -1, **i32)
        self.parent = torch.full((batch, max_nodes), -1, **i32)
        self.depth = torch.zeros((batch, max_nodes), **i32)
        self.rank = torch.full((batch, max_nodes), -1, **i32)
        self.score = torch.zeros((batch, max_nodes), **f32)
        self.n_nodes = torch.zeros((batch,), **i32)
        self.lse = torch.zeros((batch, L), **f32)
        self.cand_id = torch.zeros((batch, L, Kc), **i32)
        self.cand_lp = torch.zeros((batch, L, Kc), **f32)
        self.status = torch.zeros((batch,), **i32)

    def struct(self):
        return TreeStruct(self.max_nodes, self.Kc, self.L, *[
            _ptr(getattr(self, f)) for f in ("node_tok", "parent", "depth", "rank", "score", "n_nodes",
                                             "lse", "cand_id", "cand_lp", "status")])

    @classmethod
    def for_params(cls, p, max_nodes=None, device="cuda"):
        return cls(p.batch, p.L, p.Kc, max_nodes or p.budget + 1, device)


def workspace_size(p):
    ok = ctypes.c_int(0)
    n = lib().dt_workspace_size(ctypes.byref(p.struct(for_launch=False)), ctypes.byref(ok))
    if not ok.value:
        raise DtError("invalid parameters for dt_workspace_size")
    return int(n)


def make_workspace(p, device="cuda"):
    n = workspace_size(p)
    return torch.empty(max(n, 1), dtype=torch.uint8, device=device), n


def candidates(p, draft_logits, tree, stream=None):
    _need_logits(draft_logits, p)
    _need_batch(tree, p.batch)
    _check(lib().dt_candidates(ctypes.byref(p.struct()), _ptr(draft_logits), ctypes.byref(tree.struct()),
                               _stream(stream)), "dt_candidates")



def stage1_plan(p):
    """(kernel, cluster) that candidates() launches for Params p: kernel is
    "cluster" (each row over a cluster of `cluster` CTAs) or "rows" (a CTA per row)."""
    k, c = _i32(0), _i32(0)
    _check(lib().dt_stage1_plan(ctypes.byref(p.struct(for_launch=False)), ctypes.byref(k), ctypes.byref(c)),
           "dt_stage1_plan")
    return ({DT_STAGE1_CLUSTER: "cluster", DT_STAGE1_ROWS: "rows"}[k.value], c.value)

def stage1_ceiling(p, draft_logits, chunk_max, status=None, stream=None):
    """The read floor of the cluster stage-1 launch (dt_stage1_ceiling): every
    CTA's chunk maximum into chunk_max [batch * L, S] fp32, S from stage1_plan."""
    kind, S = stage1_plan(p)
    if kind != "cluster":
        raise DtError("dt_stage1_ceiling: the stage-1 plan for these parameters is one CTA per row")
    _need_logits(draft_logits, p)
    _need(chunk_max, torch.float32, "chunk_max", numel=p.batch * p.L * S)
    if status is not None:
        _need(status, torch.int32, "status", numel=1)
    _check(lib().dt_stage1_ceiling(ctypes.byref(p.struct()), _ptr(draft_logits), _ptr(chunk_max), _ptr(status),
                                   _stream(stream)), "dt_stage1_ceiling")


def markov_norm(p, draft_logits, tree, workspace, stream=None):
    """Full-vocabulary DARTree log-normalisers into the workspace (dt_markov_norm)."""
    _need_logits(draft_logits, p)
    _need_batch(tree, p.batch)
    ws, n = _need_workspace(workspace)
    _check(lib().dt_markov_norm(ctypes.byref(p.struct()), _ptr(draft_logits), ctypes.byref(tree.struct()), _ptr(ws),
                                n, _stream(stream)), "dt_markov_norm")


def znorm_view(p, workspace):
    """The [batch, L, K] fp32 log-normaliser table inside a DARTree workspace."""
    ws, _ = workspace
    off = (p.batch * p.L * p.K * p.K * 4 + 255) & ~255
    n = p.batch * p.L * p.K
    return ws[off:off + 4 * n].view(torch.float32).view(p.batch, p.L, p.K)


def select(p, tree, workspace=None, stream=None):
    _need_batch(tree, p.batch)
    ws, n = _need_workspace(workspace)
    _check(lib().dt_select(ctypes.byref(p.struct()), ctypes.byref(tree.struct()), _ptr(ws), n, _stream(stream)),
           "dt_select")


def select_dartree_noalloc(p, tree, stream=None):
    """DARTree selection with the library's own fixed table (no workspace);
    see dt_select_dartree_noalloc in include/dtree.h."""
    _need_batch(tree, p.batch)
    _check(lib().dt_select_dartree_noalloc(ctypes.byref(p.struct()), ctypes.byref(tree.struct()), _stream(stream)),
           "dt_select_dartree_noalloc")


def build_tree(p, draft_logits, tree, workspace=None, stream=None):
    """Stage 1 + selection.  workspace: (tensor, bytes) from make_workspace (DARTree)."""
    _need_logits(draft_logits, p)
    _need_batch(tree, p.batch)
    ws, n = _need_workspace(workspace)
    _check(lib().dt_build_tree(ctypes.byref(p.struct()), _ptr(draft_logits), ctypes.byref(tree.struct()),
                               _ptr(ws), n, _stream(stream)), "dt_build_tree")



def select_mask(p, tree, mask, pos, workspace=None, pos_offset=0, stream=None):
    """select + tree_mask with the mask written by the selection kernel (dt_select_mask)."""
    _need_batch(tree, p.batch)
    _need_mask(tree, p.batch, mask, pos)
    ws, n = _need_workspace(workspace)
    _check(lib().dt_select_mask(ctypes.byref(p.struct()), ctypes.byref(tree.struct()), _ptr(ws), n, int(pos_offset),
                                _ptr(mask), _ptr(pos), _stream(stream)), "dt_select_mask")


def build_tree_mask(p, draft_logits, tree, mask, pos, workspace=None, pos_offset=0, stream=None):
    """build_tree + tree_mask with the mask written by the selection kernel
    (dt_build_tree_mask); mask, pos from alloc_mask(tree)."""
    _need_logits(draft_logits, p)
    _need_batch(tree, p.batch)
    _need_mask(tree, p.batch, mask, pos)
    ws, n = _need_workspace(workspace)
    _check(lib().dt_build_tree_mask(ctypes.byref(p.struct()), _ptr(draft_logits), ctypes.byref(tree.struct()),
                                    _ptr(ws), n, int(pos_offset), _ptr(mask), _ptr(pos), _stream(stream)),
           "dt_build_tree_mask")

def tree_mask(tree, mask, pos, pos_offset=0, batch=None, stream=None):
    batch = batch or tree.batch
    _need_batch(tree, batch)
    _need_mask(tree, batch, mask, pos)
    _check(lib().dt_tree_mask(ctypes.byref(tree.struct()), batch, pos_offset, _ptr(mask), _ptr(pos),
                              _stream(stream)), "dt_tree_mask")


def _need_mask(tree, batch, mask, pos):
    words = (tree.max_nodes + 31) // 32
    _need(mask, torch.int32, "mask", numel=batch * tree.max_nodes * words)
    _need(pos, torch.int32, "pos", numel=batch * tree.max_nodes)


def _need_verify_io(tree, batch, V, draft, uniforms, target_lse, out, visited_lse):
    if draft is not None:
        _need(draft, name="draft", numel=batch * tree.L * V)
        if draft.shape[-1] != V:
            raise ValueError("draft rows must hold V = %d logits, got %d" % (V, draft.shape[-1]))
    if uniforms is not None:
        _need(uniforms, torch.float32, "uniforms", numel=batch * 2 * tree.max_nodes)
    if target_lse is not None:
        _need(target_lse, torch.float32, "target_lse", numel=batch * tree.max_nodes)
    acc_nodes, acc_len, next_tok = out
    _need(acc_nodes, torch.int32, "acc_nodes", numel=batch * (tree.L + 1))
    _need(acc_len, torch.int32, "acc_len", numel=batch)
    _need(next_tok, torch.int32, "next_tok", numel=batch)
    if visited_lse is not None:
        _need(visited_lse, torch.float32, "visited_lse", numel=batch * (tree.L + 1))


def alloc_mask(tree, device="cuda"):
    words = (tree.max_nodes + 31) // 32
    mask = torch.zeros((tree.batch, tree.max_nodes, words), dtype=torch.int32, device=device)
    pos = torch.zeros((tree.batch, tree.max_nodes), dtype=torch.int32, device=device)
    return mask, pos


def verify(tree, target, temperature=0.0, draft=None, uniforms=None, out=None, visited_lse=None, batch=None,
           target_lse=None, stream=None, rule=None):
    """Acceptance walk.  out = (acc_nodes [b, L+1], acc_len [b], next_tok [b]) int32 tensors;
    target_lse: optional [b, max_nodes] fp32 normalisers of the target rows (T=1);
    rule: None (greedy at temperature 0, "ratio" at 1) or one of VERIFY_RULES."""
    batch = batch or tree.batch
    _need_batch(tree, batch)
    V = target.shape[-1]
    _need(target, name="target", numel=batch * tree.max_nodes * V)
    if draft is not None and draft.dtype != target.dtype:
        # the walk reads both row sets with the target's element type
        raise TypeError("draft logits (%s) and target logits (%s) must share one dtype" % (draft.dtype, target.dtype))
    if out is None:
        with _on(stream):
            out = alloc_verify_out(tree)
    acc_nodes, acc_len, next_tok = out
    _need_verify_io(tree, batch, V, draft, uniforms, target_lse, out, visited_lse)
    if rule is not None:
        _check(lib().dt_verify_rule(ctypes.byref(tree.struct()), batch, V, _dtype_code(target), _ptr(target),
                                    _ptr(target_lse), _ptr(draft), VERIFY_RULES[rule], _ptr(uniforms),
                                    _ptr(acc_nodes), _ptr(acc_len), _ptr(next_tok), _ptr(visited_lse),
                                    _stream(stream)), "dt_verify_rule")
        return out
    _check(lib().dt_verify(ctypes.byref(tree.struct()), batch, V, _dtype_code(target), _ptr(target),
                           _ptr(target_lse), _ptr(draft), float(temperature), _ptr(uniforms), _ptr(acc_nodes),
                           _ptr(acc_len), _ptr(next_tok), _ptr(visited_lse), _stream(stream)), "dt_verify")
    return out


def verify_markov(p, tree, target, draft, znorm, uniforms, out=None, visited_lse=None, target_lse=None,
                  stream=None):
    """T=1 walk against the normalised DARTree proposal (dt_verify_markov); znorm [b, L, K] fp32,
    e.g. znorm_view(p, workspace) after markov_norm."""
    _need_batch(tree, p.batch)
    _need(target, name="target", numel=p.batch * tree.max_nodes * p.V)
    _need_logits(draft, p, "draft")
    if _dtype_code(target) != _dtype_code(draft):
        # the walk reads the target rows with the parameter block's element type
        raise TypeError("target logits must be %s for dtype=%r, got %s" % (draft.dtype, p.dtype, target.dtype))
    _need(znorm, torch.float32, "znorm", numel=p.batch * p.L * p.K)
    if out is None:
        with _on(stream):
            out = alloc_verify_out(tree)
    acc_nodes, acc_len, next_tok = out
    _need_verify_io(tree, p.batch, p.V, None, uniforms, target_lse, out, visited_lse)
    if uniforms is None:
        raise ValueError("verify_markov needs uniforms")
    _check(lib().dt_verify_markov(ctypes.byref(p.struct()), ctypes.byref(tree.struct()), _ptr(target),
                                  _ptr(target_lse), _ptr(draft), _ptr(znorm), _ptr(uniforms), _ptr(acc_nodes),
                                  _ptr(acc_len), _ptr(next_tok), _ptr(visited_lse), _stream(stream)),
           "dt_verify_markov")
    return out


def alloc_verify_out(tree, device="cuda"):
    return (torch.full((tree.batch, tree.L + 1), -1, dtype=torch.int32, device=device),
            torch.zeros((tree.batch,), dtype=torch.int32, device=device),
            torch.zeros((tree.batch,), dtype=torch.int32, device=device))


class SabaState:
    """Device SABA history for a batch: ring [batch, window] and count [batch] (int32, zeroed)."""

    def __init__(self, batch, window, device="cuda"):
        self.window = window
        self.ring = torch.zeros((batch, window), dtype=torch.int32, device=device)
        self.count = torch.zeros((batch,), dtype=torch.int32, device=device)


def saba_budget(tree, st, c_verify, c_fixed, B_min, B_max, budget, state, hidden=None, prev_acc_len=None,
                batch=None, stream=None):
    """dt_saba_budget: per-request budgets [batch] int32 and state [batch, 4] fp32 (conf, degen, hist, a);
    hidden: optional [batch, L, Hd] fp32 drafter hidden states; prev_acc_len: last round's acc_len."""
    batch = batch or tree.batch
    _need_batch(tree, batch)
    _need(budget, torch.int32, "budget", numel=batch)
    _need(state, torch.float32, "state", numel=batch * 4)
    _need(st.ring, torch.int32, "ring", numel=batch * st.window)
    _need(st.count, torch.int32, "count", numel=batch)
    Hd = 0
    if hidden is not None:
        Hd = int(hidden.shape[-1])
        _need(hidden, torch.float32, "hidden", numel=batch * tree.L * Hd)
    if prev_acc_len is not None:
        _need(prev_acc_len, torch.int32, "prev_acc_len", numel=batch)
    q = SabaStruct(st.window, float(c_verify), float(c_fixed), int(B_min), int(B_max))
    _check(lib().dt_saba_budget(ctypes.byref(q), ctypes.byref(tree.struct()), batch, _ptr(hidden), Hd,
                                _ptr(prev_acc_len), _ptr(st.ring), _ptr(st.count), _ptr(state), _ptr(budget),
                                _stream(stream)), "dt_saba_budget")


# ---------------------------------------------------------------------------
# The target model's side of a round: norms of its heads, paged caches in e4m3 or 4 bits,
# tree attention over them, and log-probabilities of what was emitted.
# ---------------------------------------------------------------------------

class PagedCache:
    """Keys and values in pages of e4m3 numbers with a scale per (page, key head) (dt_kv_cache).

    k, v: [n_pages, Hkv, page, D] uint8 (or float8_e4m3fn) codes; k_scale, v_scale: [n_pages, Hkv] fp32;
    table: [batch, max_pages] int32; len: [batch] int32 tokens held.  The caller owns all of them and
    assigns pages by writing `table`; reassigning an attribute needs a new PagedCache."""

    def __init__(self, k, v, k_scale, v_scale, table, len):
        if k.dim() != 4 or k.shape != v.shape:
            raise ValueError("k and v must be [n_pages, Hkv, page, D] of one shape, got %s and %s"
                             % (tuple(k.shape), tuple(v.shape)))
        for t, name in ((k, "k"), (v, "v")):
            _need(t, name=name)
            if t.dtype not in (torch.uint8, torch.float8_e4m3fn):
                raise TypeError("%s must be uint8 or float8_e4m3fn codes, got %s" % (name, t.dtype))
        self.n_pages, self.Hkv, self.page, self.D = k.shape
        _need(k_scale, torch.float32, "k_scale", numel=self.n_pages * self.Hkv)
        _need(v_scale, torch.float32, "v_scale", numel=self.n_pages * self.Hkv)
        _need(table, torch.int32, "table")
        if table.dim() != 2:
            raise ValueError("table must be [batch, max_pages], got %s" % (tuple(table.shape),))
        self.batch, self.max_pages = table.shape
        _need(len, torch.int32, "len", numel=self.batch)
        if {t.get_device() for t in (k, v, k_scale, v_scale, len)} != {table.get_device()}:
            raise ValueError("a cache's tensors must be on one device")
        self.k, self.v, self.k_scale, self.v_scale, self.table, self.len = k, v, k_scale, v_scale, table, len
        self._struct = CacheStruct(self.n_pages, self.page, self.Hkv, self.D, self.max_pages, k.data_ptr(),
                                   v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), table.data_ptr(),
                                   len.data_ptr())
        self._ref = ctypes.byref(self._struct)
        self._device = table.get_device()

    @classmethod
    def empty(cls, n_pages, page, Hkv, D, batch, max_pages, device="cuda"):
        """A cache with nothing in it: every length 0, every table entry -1."""
        u8 = dict(dtype=torch.uint8, device=device)
        f32 = dict(dtype=torch.float32, device=device)
        i32 = dict(dtype=torch.int32, device=device)
        return cls(torch.zeros((n_pages, Hkv, page, D), **u8), torch.zeros((n_pages, Hkv, page, D), **u8),
                   torch.ones((n_pages, Hkv), **f32), torch.ones((n_pages, Hkv), **f32),
                   torch.full((batch, max_pages), -1, **i32), torch.zeros((batch,), **i32))


class PagedCache4:
    """Keys and values in pages of e2m1 numbers, 4.5 bits an element (dt_kv_cache4): append, attention and
    reading take it in place of a PagedCache.

    k, v: [n_pages, Hkv, page, D / 2] uint8 codes, element 2i in the lower half of byte i; k_scale, v_scale:
    [n_pages, Hkv, page, D / 16] uint8, a scale for each 16 elements (the upper half of an fp16 number without
    its sign); table: [batch, max_pages] int32; len: [batch] int32.  The caller owns all of them, as there."""

    def __init__(self, k, v, k_scale, v_scale, table, len):
        if k.dim() != 4 or k.shape != v.shape:
            raise ValueError("k and v must be [n_pages, Hkv, page, D / 2] of one shape, got %s and %s"
                             % (tuple(k.shape), tuple(v.shape)))
        self.n_pages, self.Hkv, self.page, self.D = *k.shape[:3], 2 * k.shape[3]
        for t, name in ((k, "k"), (v, "v"), (k_scale, "k_scale"), (v_scale, "v_scale")):
            _need(t, torch.uint8, name)
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t.shape != (*k.shape[:3], self.D // 16):
                raise ValueError("%s must be %s, got %s" % (name, (*k.shape[:3], self.D // 16), tuple(t.shape)))
        _need(table, torch.int32, "table")
        if table.dim() != 2:
            raise ValueError("table must be [batch, max_pages], got %s" % (tuple(table.shape),))
        self.batch, self.max_pages = table.shape
        _need(len, torch.int32, "len", numel=self.batch)
        if {t.get_device() for t in (k, v, k_scale, v_scale, len)} != {table.get_device()}:
            raise ValueError("a cache's tensors must be on one device")
        self.k, self.v, self.k_scale, self.v_scale, self.table, self.len = k, v, k_scale, v_scale, table, len
        self._struct = CacheStruct(self.n_pages, self.page, self.Hkv, self.D, self.max_pages, k.data_ptr(),
                                   v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), table.data_ptr(),
                                   len.data_ptr())
        self._ref = ctypes.byref(self._struct)
        self._device = table.get_device()

    @classmethod
    def empty(cls, n_pages, page, Hkv, D, batch, max_pages, device="cuda"):
        """A cache with nothing in it: every length 0, every table entry -1."""
        u8 = dict(dtype=torch.uint8, device=device)
        i32 = dict(dtype=torch.int32, device=device)
        return cls(torch.zeros((n_pages, Hkv, page, D // 2), **u8), torch.zeros((n_pages, Hkv, page, D // 2), **u8),
                   torch.zeros((n_pages, Hkv, page, D // 16), **u8), torch.zeros((n_pages, Hkv, page, D // 16), **u8),
                   torch.full((batch, max_pages), -1, **i32), torch.zeros((batch,), **i32))


class Rope:
    """Rotation tables (dt_rope): cos, sin [max_pos, rot / 2] fp32."""

    def __init__(self, cos, sin, interleaved=False):
        _need(cos, torch.float32, "cos")
        _need(sin, torch.float32, "sin", numel=cos.numel())
        if cos.dim() != 2 or cos.shape != sin.shape:
            raise ValueError("cos and sin must be [max_pos, rot / 2], got %s and %s"
                             % (tuple(cos.shape), tuple(sin.shape)))
        self.cos, self.sin, self.interleaved = cos, sin, bool(interleaved)
        self._struct = RopeStruct(cos.data_ptr(), sin.data_ptr(), cos.shape[0], 2 * cos.shape[1], int(self.interleaved))
        self._ref = ctypes.byref(self._struct)
        self._device = cos.get_device()


def _head_rows(t, shape, name, device):
    """dt_rows of [batch, M, H, D]: any strides with dense, 16-byte aligned head vectors.
    device: the current one (torch.cuda.current_device(), read once per call)."""
    if t.get_device() != device:
        raise ValueError("%s must be a CUDA tensor on the current device" % name)
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, shape, tuple(t.shape)))
    sb, sn, sh, sd = t.stride()
    if sd != 1:
        raise ValueError("%s must be dense in its last dimension" % name)
    return RowsStruct(t.data_ptr(), sb, sn, sh)


def _need_here(x, name, device):
    """A cache or rotation tables on the current device (None: nothing to check)."""
    if x is not None and x._device != device:
        raise ValueError("%s must be on the current device" % name)


def _need_at(t, device, dtype, name, numel=None):
    """_need on the current device."""
    if t.get_device() == device and t.is_contiguous() and t.dtype == dtype and (numel is None or t.numel() >= numel):
        return t
    if t.is_cuda and t.get_device() != device:
        raise ValueError("%s must be on the current device" % name)
    return _need(t, dtype, name, numel)


def _addr(t):
    return None if t is None else t.data_ptr()


class Pair(tuple):
    """Two tensors that a call returns, and as `.status` the status words that it set: the caller's, or, when
    it brought none, the call's own."""
    status = None


def _pair(a, b, status):
    pair = Pair((a, b))
    pair.status = status
    return pair


def kv_append(cache, k, v, rope=None, rows=None, count=None, count_add=0, len_out=None, status=None, stream=None):
    """Append rows of k, v [batch, M, Hkv, D] to the cache (dt_kv_append, dt_kv_append4): keys rotated to
    their position on the way, both stored in the cache's form.  rows [batch, N] int32 picks rows (the walk's acc_nodes),
    count [batch] int32 + count_add says how many (its acc_len, 1); len_out [batch] gets the new lengths;
    status [batch] int32 is OR-ed with DT_DEV_BAD_CACHE for a request that does not fit; returned."""
    batch, M, device = cache.batch, k.shape[1], torch.cuda.current_device()
    _need_here(cache, "cache", device)
    _need_here(rope, "rope", device)
    if k.dtype != v.dtype:
        raise TypeError("k (%s) and v (%s) must share one dtype" % (k.dtype, v.dtype))
    shape = (batch, M, cache.Hkv, cache.D)
    kr, vr = _head_rows(k, shape, "k", device), _head_rows(v, shape, "v", device)
    N = M
    if rows is not None:
        _need_at(rows, device, torch.int32, "rows")
        if rows.dim() != 2 or rows.shape[0] != batch:
            raise ValueError("rows must be [batch, N], got %s" % (tuple(rows.shape),))
        N = rows.shape[1]
    if count is not None:
        _need_at(count, device, torch.int32, "count", numel=batch)
    if len_out is not None:
        _need_at(len_out, device, torch.int32, "len_out", numel=batch)
    if status is None:
        with _on(stream):
            status = torch.zeros((batch,), dtype=torch.int32, device=k.device)
    else:
        _need_at(status, device, torch.int32, "status", numel=batch)
    call = lib().dt_kv_append4 if isinstance(cache, PagedCache4) else lib().dt_kv_append
    _check(call(cache._ref, rope._ref if rope is not None else None, batch, M, _dtype_code(k), kr, vr, _addr(rows), N,
                _addr(count), int(count_add), _addr(len_out), status.data_ptr(),
                _raw_stream(device) if stream is None else stream.cuda_stream), "dt_kv_append")
    return status


def kv_read(cache, N=None, rows=None, start=None, count=None, count_add=0, dtype=torch.bfloat16, k=None, v=None,
            status=None, stream=None):
    """Read tokens back out of a PagedCache or PagedCache4 (dt_kv_read, dt_kv_read4): row j of request b is
    token rows[b, j] (rows [batch, N] int32), or start[b] + j (start [batch] int32; None: 0).
    count [batch] int32 + count_add says how many rows a request gets, in [0, N]; without it, all of `rows`,
    or all tokens from start on.  k, v: outputs [batch, N, Hkv, D] bf16 or fp32, any strides with dense heads
    (None: zeros of `dtype`; N is needed then when there are no rows).  status [batch] int32 (None: made here) is
    OR-ed with DT_DEV_BAD_CACHE for a request out of range, which is left alone as a whole: its rows stay zeros in
    outputs made here.  Returns (k, v), with the status words as `.status`."""
    batch, Hkv, D, device = cache.batch, cache.Hkv, cache.D, torch.cuda.current_device()
    _need_here(cache, "cache", device)
    if rows is not None:
        _need_at(rows, device, torch.int32, "rows")
        if rows.dim() != 2 or rows.shape[0] != batch:
            raise ValueError("rows must be [batch, N], got %s" % (tuple(rows.shape),))
        if start is not None:
            raise ValueError("rows and start exclude each other")
    for x in (rows, k, v):
        if x is None:
            continue
        if N is None:
            N = x.shape[1]
        if x.shape[1] != N:
            raise ValueError("N, rows and outputs speak of %d and %d rows" % (N, x.shape[1]))
    if N is None:
        raise ValueError("N is needed without rows and outputs")
    if start is not None:
        _need_at(start, device, torch.int32, "start", numel=batch)
    if count is not None:
        _need_at(count, device, torch.int32, "count", numel=batch)
    if k is None or v is None or status is None:
        with _on(stream):
            held = dict(dtype=dtype if k is None and v is None else (v if k is None else k).dtype, device=cache.k.device)
            if k is None:
                k = torch.zeros((batch, N, Hkv, D), **held)
            if v is None:
                v = torch.zeros((batch, N, Hkv, D), **held)
            if status is None:
                status = torch.zeros((batch,), dtype=torch.int32, device=cache.k.device)
    _need_at(status, device, torch.int32, "status", numel=batch)
    if k.dtype != v.dtype:
        raise TypeError("k (%s) and v (%s) must share one dtype" % (k.dtype, v.dtype))
    shape = (batch, N, Hkv, D)
    kr, vr = _head_rows(k, shape, "k", device), _head_rows(v, shape, "v", device)
    call = lib().dt_kv_read4 if isinstance(cache, PagedCache4) else lib().dt_kv_read
    _check(call(cache._ref, batch, _addr(rows), N, _addr(start), _addr(count), int(count_add), _dtype_code(k), kr, vr,
                status.data_ptr(), _raw_stream(device) if stream is None else stream.cuda_stream), "dt_kv_read")
    return _pair(k, v, status)


def _norm_weight(w, H, D, name, device):
    """(address, stride between heads) of weights [D] or [H, D]."""
    if w is None:
        return None, 0
    _need_at(w, device, torch.float32, name)
    if w.shape not in ((D,), (H, D)):
        raise ValueError("%s must be %s or %s, got %s" % (name, (D,), (H, D), tuple(w.shape)))
    return w.data_ptr(), D if w.dim() == 2 else 0


def qk_norm(q, k, q_weight=None, k_weight=None, eps=1e-6, rope=None, len=None, pos=None, n_nodes=None, q_out=None,
            k_out=None, status=None, stream=None):
    """Root-mean-square norms of query and key heads, rotated in the same pass (dt_qk_norm): q [batch, M, Hq, D],
    k [batch, M, Hk, D] bf16 or fp32 (k None: queries alone); weights fp32 [D] or [heads, D] (None: ones).
    Row n of request b has position len[b] + pos[b, n] (len None: 0; pos None: n).  Outputs are like q and k and
    may be q and k themselves; rows from n_nodes[b] on are left alone in outputs that the caller brings, and
    undefined in others; so are rows whose position is out of range, and all of a request whose count is.
    tree_attention and kv_append then take the results with rope None.  status [batch] int32 (None: made here) is
    OR-ed with DT_DEV_BAD_CACHE for such a request.  Returns (q_out, k_out), with the status words as `.status`."""
    batch, M, Hq, D = q.shape
    Hk, device, dtype = 0 if k is None else k.shape[2], torch.cuda.current_device(), q.dtype
    _need_here(rope, "rope", device)
    if k is None and k_out is not None:
        raise ValueError("k_out needs k")
    if q_out is None or (k_out is None and k is not None) or status is None:
        with _on(stream):
            if q_out is None:
                q_out = torch.empty((batch, M, Hq, D), dtype=q.dtype, device=q.device)
            if k_out is None and k is not None:
                k_out = torch.empty((batch, M, Hk, D), dtype=q.dtype, device=q.device)
            if status is None:
                status = torch.zeros((batch,), dtype=torch.int32, device=q.device)
    shape = (batch, M, Hq, D)
    qr, qo = _head_rows(q, shape, "q", device), _head_rows(q_out, shape, "q_out", device)
    kr = ko = None
    if q_out.dtype != dtype:
        raise TypeError("q_out must be %s, got %s" % (dtype, q_out.dtype))
    if k is not None:
        shape = (batch, M, Hk, D)
        kr, ko = _head_rows(k, shape, "k", device), _head_rows(k_out, shape, "k_out", device)
        if k.dtype != dtype or k_out.dtype != dtype:
            raise TypeError("k and k_out must be %s, got %s and %s" % (dtype, k.dtype, k_out.dtype))
    if len is not None:
        _need_at(len, device, torch.int32, "len", numel=batch)
    if pos is not None:
        _need_at(pos, device, torch.int32, "pos", numel=batch * M)
    if n_nodes is not None:
        _need_at(n_nodes, device, torch.int32, "n_nodes", numel=batch)
    _need_at(status, device, torch.int32, "status", numel=batch)
    qw, qs = _norm_weight(q_weight, Hq, D, "q_weight", device)
    kw, ks = _norm_weight(k_weight, Hk, D, "k_weight", device)
    _check(lib().dt_qk_norm(batch, M, Hq, Hk, D, _dtype_code(q), qr, kr, qw, qs, kw, ks, eps,
                            rope._ref if rope is not None else None, _addr(len), _addr(pos), _addr(n_nodes), qo, ko,
                            status.data_ptr(), _raw_stream(device) if stream is None else stream.cuda_stream), "dt_qk_norm")
    return _pair(q_out, k_out, status)


def attention_workspace(cache, M, Hq):
    """Zeroed workspace of tree_attention calls on this cache with M rows and Hq query heads (or
    fewer of either): (tensor, bytes).  Calls that may run at the same time need one each."""
    size = lib().dt_tree_attention4_workspace if isinstance(cache, PagedCache4) else lib().dt_tree_attention_workspace
    n = int(size(cache._ref, cache.batch, M, Hq))
    return torch.zeros(max(n, 16), dtype=torch.uint8, device=cache.k.device), n


def tree_attention(cache, q, k, v, mask=None, pos=None, n_nodes=None, rope=None, scale=None, out=None, workspace=None,
                   status=None, stream=None):
    """Attention of the tree's rows over the cache and over the tree (dt_tree_attention, dt_tree_attention4).
    q [batch, M, Hq, D], k, v [batch, M, Hkv, D] bf16, not rotated; mask, pos as dt_tree_mask writes
    them with pos_offset 0 (None: a chain); returns out [batch, M, Hq, D] bf16.  status [batch] int32
    is OR-ed with DT_DEV_BAD_CACHE for a request out of range: bring one to see it."""
    batch, M, Hq, device = cache.batch, q.shape[1], q.shape[2], torch.cuda.current_device()
    _need_here(cache, "cache", device)
    _need_here(rope, "rope", device)
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        if t.dtype != torch.bfloat16:
            raise TypeError("%s must be bfloat16, got %s" % (name, t.dtype))
    qr = _head_rows(q, (batch, M, Hq, cache.D), "q", device)
    shape = (batch, M, cache.Hkv, cache.D)
    kr, vr = _head_rows(k, shape, "k", device), _head_rows(v, shape, "v", device)
    if mask is not None:
        _need_at(mask, device, torch.int32, "mask", numel=batch * M * ((M + 31) // 32))
    if pos is not None:
        _need_at(pos, device, torch.int32, "pos", numel=batch * M)
    if n_nodes is not None:
        _need_at(n_nodes, device, torch.int32, "n_nodes", numel=batch)
    if out is not None:
        _need_at(out, device, torch.bfloat16, "out", numel=batch * M * Hq * cache.D)
    if status is not None:
        _need_at(status, device, torch.int32, "status", numel=batch)
    if out is None or status is None or workspace is None:
        with _on(stream):
            if out is None:
                out = torch.empty((batch, M, Hq, cache.D), dtype=torch.bfloat16, device=q.device)
            if status is None:
                status = torch.zeros((batch,), dtype=torch.int32, device=q.device)
            if workspace is None:
                workspace = attention_workspace(cache, M, Hq)
    ws, n = _need_workspace(workspace)
    if ws is not None and ws.get_device() != device:
        raise ValueError("workspace must be on the current device")
    if scale is None:
        scale = 1.0 / math.sqrt(cache.D)
    call = lib().dt_tree_attention4 if isinstance(cache, PagedCache4) else lib().dt_tree_attention
    _check(call(cache._ref, rope._ref if rope is not None else None, batch, M, Hq, qr, kr, vr, _addr(mask), _addr(pos),
                _addr(n_nodes), scale, out.data_ptr(), _addr(ws), n, status.data_ptr(),
                _raw_stream(device) if stream is None else stream.cuda_stream), "dt_tree_attention")
    return out


@dataclasses.dataclass
class Logprobs:
    """Outputs of token_logprobs: logprob, entropy [batch, N] fp32, rank [batch, N] int32, and
    top_id int32, top_logprob fp32 [batch, N, top] (None when top is 0)."""
    logprob: torch.Tensor
    entropy: torch.Tensor
    rank: torch.Tensor
    top_id: torch.Tensor = None
    top_logprob: torch.Tensor = None


def alloc_logprobs(batch, N, top=0, device="cuda"):
    f32 = dict(dtype=torch.float32, device=device)
    i32 = dict(dtype=torch.int32, device=device)
    o = Logprobs(torch.zeros((batch, N), **f32), torch.zeros((batch, N), **f32), torch.full((batch, N), -1, **i32))
    if top > 0:
        o.top_id, o.top_logprob = torch.full((batch, N, top), -1, **i32), torch.zeros((batch, N, top), **f32)
    return o


def token_logprobs(logits, tokens, top=0, rows=None, out=None, stream=None):
    """Log-probability, rank and entropy for tokens [batch, N] int32 under rows of logits [batch, M, V]
    (row j, or rows[b, j]), with the `top` best alternatives (dt_token_logprobs).  Negative entries
    of rows or tokens are padding."""
    if logits.dim() != 3 or not logits.is_cuda:
        raise ValueError("logits must be a CUDA tensor [batch, M, V]")
    batch, M, V = logits.shape
    sb, sm, sv = logits.stride()
    if sv != 1 and V > 1 or sm < V and M > 1:
        raise ValueError("logits must be dense in V and their rows apart, got strides %s" % (logits.stride(),))
    _need(tokens, torch.int32, "tokens")
    if tokens.dim() != 2 or tokens.shape[0] != batch:
        raise ValueError("tokens must be [batch, N], got %s" % (tuple(tokens.shape),))
    N = tokens.shape[1]
    if rows is not None:
        _need(rows, torch.int32, "rows")
        if rows.shape != tokens.shape:
            raise ValueError("rows must be shaped as tokens, got %s and %s" % (tuple(rows.shape), tuple(tokens.shape)))
    if out is None:
        with _on(stream):
            out = alloc_logprobs(batch, N, top, logits.device)
    else:
        _need(out.logprob, torch.float32, "logprob", numel=batch * N)
        _need(out.entropy, torch.float32, "entropy", numel=batch * N)
        _need(out.rank, torch.int32, "rank", numel=batch * N)
        if top > 0:
            if out.top_id is None or out.top_logprob is None:
                raise ValueError("out has no room for alternatives (alloc_logprobs(batch, N, top))")
            _need(out.top_id, torch.int32, "top_id", numel=batch * N * top)
            _need(out.top_logprob, torch.float32, "top_logprob", numel=batch * N * top)
    _check(lib().dt_token_logprobs(_addr(logits), _dtype_code(logits), batch, M, V, sb, max(sm, V), _addr(rows),
                                   _addr(tokens), N, int(top), _addr(out.logprob), _addr(out.entropy), _addr(out.rank),
                                   _addr(out.top_id) if top > 0 else None, _addr(out.top_logprob) if top > 0 else None,
                                   _stream(stream)), "dt_token_logprobs")
    return out
