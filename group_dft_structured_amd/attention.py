"""Binding of attention over packed sequences (``include/eqattn.h``): argument
marshalling only."""
import ctypes
import functools
import math
from array import array

from . import _DTYPE_CODE, EQL_F16, _check, _ptr, _stream, load_library
from ._tensors import Launch, expect, expect_rows, expect_workspace, refuse, torch_dtype

ATTN_EXPORTED = (
    "eqattn_plan_create",
    "eqattn_plan_destroy",
    "eqattn_forward_workspace",
    "eqattn_forward",
    "eqattn_backward_workspace",
    "eqattn_backward_workspace_no_dtable",
    "eqattn_backward",
)


class View(ctypes.Structure):
    """eqattn_view_t: first element, and strides in elements."""
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class PackingStruct(ctypes.Structure):
    """eqattn_packing_t."""
    _fields_ = [(n, ctypes.c_int64) for n in ("sequences", "total_q", "total_k", "max_q", "max_k")] \
        + [(n, ctypes.c_void_p) for n in ("cu_q", "cu_k", "pos_q", "pos_k")]


@functools.lru_cache(None)
def _lib():
    lib = load_library()
    vp, i64, st, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    view = pack = vp  # addresses of structures
    lib.eqattn_plan_create.argtypes = [i64, i64, i64, ctypes.c_double, st, i64, i64, st,
                                       ctypes.POINTER(vp)]
    lib.eqattn_plan_create.restype = st
    lib.eqattn_plan_destroy.argtypes = [vp]
    lib.eqattn_plan_destroy.restype = st
    lib.eqattn_forward_workspace.argtypes = [vp, pack]
    lib.eqattn_forward_workspace.restype = sz
    lib.eqattn_forward.argtypes = [vp, pack, view, view, view, vp, vp, view, vp, vp, sz, vp]
    lib.eqattn_forward.restype = st
    lib.eqattn_backward_workspace.argtypes = [vp, pack]
    lib.eqattn_backward_workspace.restype = sz
    lib.eqattn_backward_workspace_no_dtable.argtypes = [vp, pack]
    lib.eqattn_backward_workspace_no_dtable.restype = sz
    lib.eqattn_backward.argtypes = [vp, pack] + [view] * 5 + [vp, vp, vp] + [view] * 3 + \
        [vp, vp, sz, vp]
    lib.eqattn_backward.restype = st
    return lib


# --------------------------------------------------------------------------
# C ABI, one function per entry point (same names).  packing: a PackingStruct or
# its address; views: View structures or their addresses.

def _at(struct):
    return struct if struct is None or isinstance(struct, int) else ctypes.addressof(struct)


def eqattn_plan_create(heads, kv_heads, dim, scale, causal=False, buckets=0, span=0,
                       dtype=EQL_F16):
    h = ctypes.c_void_p()
    _check(_lib().eqattn_plan_create(heads, kv_heads, dim, scale, int(causal), buckets, span, dtype,
                                     ctypes.byref(h)), "eqattn_plan_create")
    return h.value


def eqattn_plan_destroy(plan):
    _check(_lib().eqattn_plan_destroy(plan), "eqattn_plan_destroy")


def eqattn_forward_workspace(plan, packing):
    return int(_lib().eqattn_forward_workspace(plan, _at(packing)))


def eqattn_forward(plan, packing, q, k, v, table, bucket_map, o, lse, workspace, workspace_bytes,
                   stream=None):
    _check(_lib().eqattn_forward(plan, _at(packing), _at(q), _at(k), _at(v), _ptr(table),
                                 _ptr(bucket_map), _at(o), _ptr(lse), _ptr(workspace), workspace_bytes, _stream(stream)),
           "eqattn_forward")


def eqattn_backward_workspace(plan, packing):
    return int(_lib().eqattn_backward_workspace(plan, _at(packing)))


def eqattn_backward_workspace_no_dtable(plan, packing):
    return int(_lib().eqattn_backward_workspace_no_dtable(plan, _at(packing)))


def eqattn_backward(plan, packing, dout, q, k, v, o, lse, table, bucket_map, dq, dk, dv, dtable,
                    workspace, workspace_bytes, stream=None):
    _check(_lib().eqattn_backward(plan, _at(packing), _at(dout), _at(q), _at(k), _at(v), _at(o),
                                  _ptr(lse), _ptr(table), _ptr(bucket_map), _at(dq), _at(dk),
                                  _at(dv), _ptr(dtable), _ptr(workspace), workspace_bytes,
                                  _stream(stream)), "eqattn_backward")


# --------------------------------------------------------------------------
# Convenience wrapper over torch tensors (still only marshalling).

class Packing:
    """How the tokens of a call are packed into sequences.

    cu_q [sequences + 1]: int32 CUDA tensor of token offsets; max_q: the longest
    sequence (a host number, so that no call waits for the GPU).  cu_k and max_k
    default to the queries'.  pos_q and pos_k: int32 positions of the tokens
    (None: the index in the sequence, queries at the end of the keys)."""

    def __init__(self, cu_q, max_q, cu_k=None, max_k=None, pos_q=None, pos_k=None):
        self.cu_q, self.max_q = cu_q, max_q
        self.cu_k = cu_q if cu_k is None else cu_k
        self.max_k = max_q if max_k is None else max_k
        self.pos_q, self.pos_k = pos_q, pos_k
        if pos_k is None and cu_k is None:
            self.pos_k = pos_q

    def fields(self, total_q, total_k, go):
        """The fields of eqattn_packing_t for these token counts, tensors checked."""
        i32, dev = go.torch.int32, go.device
        rows = self.cu_q.shape
        if len(rows) != 1 or rows[0] < 1:
            refuse(self.cu_q, ("sequences + 1",), i32, dev, "contiguous ")
        cq = expect(self.cu_q, rows, i32, dev)
        ck = cq if self.cu_k is self.cu_q else expect(self.cu_k, rows, i32, dev)
        pq = 0 if self.pos_q is None else expect(self.pos_q, (total_q,), i32, dev)
        pk = 0 if self.pos_k is None else expect(self.pos_k, (total_k,), i32, dev)
        return rows[0] - 1, total_q, total_k, self.max_q, self.max_k, cq, ck, pq, pk


_PACKING, _VIEW = 8 * 9, 8 * 3  # bytes of the structures: int64 fields and addresses


class AttnPlan:
    """Attention over packed sequences; calls take torch CUDA tensors
    [tokens, heads, dim] whose last axis is contiguous (parts of a larger tensor
    are fine), and with a bias (buckets > 0) table [buckets, heads] and
    bucket_map [2 span + 1] int32.  scale defaults to 1 / sqrt(dim)."""

    def __init__(self, heads, dim, kv_heads=None, dtype="f16", causal=False, scale=None, buckets=0,
                 span=0):
        self.handle = None
        self.H, self.Hk, self.dim, self.dtype = heads, heads if kv_heads is None else kv_heads, dim, dtype
        self.causal, self.buckets, self.span = causal, buckets, span
        self.scale = 1.0 / math.sqrt(dim) if scale is None else scale
        self._dt = torch_dtype(dtype)
        self.handle = eqattn_plan_create(self.H, self.Hk, dim, self.scale, causal, buckets, span,
                                         _DTYPE_CODE[dtype])

    def close(self):
        if self.handle:
            eqattn_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:  # noqa: BLE001 -- interpreter shutdown
            pass

    def _bias(self, table, bucket_map, go):
        if table is None and bucket_map is None:
            return None, None  # the library refuses that of a plan with a bias
        return (None if table is None else
                expect(table, (self.buckets, self.H), self._dt, go.device),
                None if bucket_map is None else
                expect(bucket_map, (2 * self.span + 1,), go.torch.int32, go.device))

    def forward(self, q, k, v, packing, table=None, bucket_map=None, o=None, lse=None,
                workspace=None, stream=None, want_lse=True):
        """(o, lse): o like q (contiguous), lse binary32 [heads, total_q] for the
        backward pass (want_lse=False: only if given)."""
        go, dt = Launch(stream), self._dt
        dev, nq, nk = go.device, q.shape[0], k.shape[0]
        qs, ks = (nq, self.H, self.dim), (nk, self.Hk, self.dim)
        views = (*expect_rows(q, qs, dt, dev), *expect_rows(k, ks, dt, dev), *expect_rows(v, ks, dt, dev))
        if o is None:
            o = go.like(q)
            po = o.data_ptr(), self.H * self.dim, self.dim
        else:
            po = expect_rows(o, qs, dt, dev)
        # the packing and the views as the C structures lie in memory
        a = array("q", (*packing.fields(nq, nk, go), *views, *po))
        pk = a.buffer_info()[0]
        vq = pk + _PACKING
        pt, pm = self._bias(table, bucket_map, go)
        pl = None
        if lse is not None:
            pl = expect(lse, (self.H, nq), go.torch.float32, dev)
        elif want_lse:
            lse = go.empty((self.H, nq), go.torch.float32)
            pl = lse.data_ptr()
        lib, pw = _lib(), None
        if workspace is not None:
            pw, nbytes = expect_workspace(workspace, dev)
        else:
            nbytes = lib.eqattn_forward_workspace(self.handle, pk)
            if nbytes:
                workspace = go.empty((nbytes,), go.torch.uint8)
                pw = workspace.data_ptr()
        st = lib.eqattn_forward(self.handle, pk, vq, vq + _VIEW, vq + 2 * _VIEW, pt, pm,
                                vq + 3 * _VIEW, pl, pw, nbytes, go.address)
        if st:
            _check(st, "eqattn_forward")
        return o, lse

    def workspace_bytes(self, packing, total_q, total_k):
        """(forward, backward) workspace bytes, for a backward pass with dtable."""
        a = array("q", packing.fields(total_q, total_k, Launch(None)))
        pk = a.buffer_info()[0]
        return (eqattn_forward_workspace(self.handle, pk),
                eqattn_backward_workspace(self.handle, pk))

    def backward(self, dout, q, k, v, o, lse, packing, table=None, bucket_map=None, dq=None, dk=None,
                 dv=None, dtable=None, workspace=None, stream=None, want_table=True):
        """(dq, dk, dv, dtable); dtable binary32 [buckets, heads] (None without a
        bias; want_table=False: only if given)."""
        go, dt = Launch(stream), self._dt
        f32, dev, nq, nk = go.torch.float32, go.device, q.shape[0], k.shape[0]
        qs, ks = (nq, self.H, self.dim), (nk, self.Hk, self.dim)
        dq = go.empty(qs, dt) if dq is None else dq
        dk = go.empty(ks, dt) if dk is None else dk
        dv = go.empty(ks, dt) if dv is None else dv
        a = array("q", (*packing.fields(nq, nk, go), *expect_rows(dout, qs, dt, dev),
                        *expect_rows(q, qs, dt, dev), *expect_rows(k, ks, dt, dev),
                        *expect_rows(v, ks, dt, dev), *expect_rows(o, qs, dt, dev),
                        *expect_rows(dq, qs, dt, dev), *expect_rows(dk, ks, dt, dev),
                        *expect_rows(dv, ks, dt, dev)))
        pk = a.buffer_info()[0]
        views = [pk + _PACKING + _VIEW * i for i in range(8)]
        pl = expect(lse, (self.H, nq), f32, dev)
        pt, pm = self._bias(table, bucket_map, go)
        if dtable is None and want_table and self.buckets:
            dtable = go.empty((self.buckets, self.H), f32)
        pd = None if dtable is None else expect(dtable, (self.buckets, self.H), f32, dev)
        lib = _lib()
        if workspace is not None:
            pw, nbytes = expect_workspace(workspace, dev)
        else:
            size = lib.eqattn_backward_workspace_no_dtable if pd is None else lib.eqattn_backward_workspace
            nbytes = size(self.handle, pk)
            workspace = go.empty((nbytes,), go.torch.uint8)
            pw = workspace.data_ptr()
        st = lib.eqattn_backward(self.handle, pk, *views[:5], pl, pt, pm, *views[5:], pd, pw, nbytes,
                                 go.address)
        if st:
            _check(st, "eqattn_backward")
        return dq, dk, dv, dtable
