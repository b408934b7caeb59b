"""The linear layer's products and the Muon and AdamW steps (include/ddl.h).

Argument checks and marshalling only.  Arrays are torch tensors on the GPU (or
objects like them); streams as elsewhere (None = the null stream).
"""
import ctypes

from ._ddl import DDL_F16, DDL_F32, _check, _ptr, lib

DDL_BF16 = 2
ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
_LINEAR_OPS = {"forward": 0, "dgrad": 1, "wgrad": 2}
_TYPES = {"torch.float32": DDL_F32, "torch.float16": DDL_F16, "torch.bfloat16": DDL_BF16}
NORM_EPS = 1e-7  # added to the norm before Muon's first product


class ddl_linear_args(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_size_t) for n in "mnk"] + [("dtype", ctypes.c_int),
                                                         ("act", ctypes.c_int)]
                + [("x", ctypes.c_void_p), ("ldx", ctypes.c_size_t), ("w", ctypes.c_void_p),
                   ("ldw", ctypes.c_size_t), ("bias", ctypes.c_void_p),
                   ("residual", ctypes.c_void_p), ("ldr", ctypes.c_size_t),
                   ("y", ctypes.c_void_p), ("ldy", ctypes.c_size_t), ("z", ctypes.c_void_p),
                   ("ldz", ctypes.c_size_t)])


class ddl_dgrad_args(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_size_t) for n in "mnk"] + [("dtype", ctypes.c_int),
                                                         ("act", ctypes.c_int)]
                + [(n, t) for p, ld in (("dz", "lddz"), ("w", "ldw"), ("residual", "ldr"),
                                        ("dx", "lddx"), ("z_prev", "ldz_prev"),
                                        ("dz_prev", "lddz_prev"))
                   for n, t in ((p, ctypes.c_void_p), (ld, ctypes.c_size_t))])


class ddl_wgrad_args(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_size_t) for n in "mnk"]
                + [(n, ctypes.c_int) for n in ("dtype", "out_dtype", "accumulate")]
                + [("dz", ctypes.c_void_p), ("lddz", ctypes.c_size_t), ("x", ctypes.c_void_p),
                   ("ldx", ctypes.c_size_t), ("dw", ctypes.c_void_p), ("lddw", ctypes.c_size_t),
                   ("db", ctypes.c_void_p)])


class ddl_muon_matrix(ctypes.Structure):
    _fields_ = [("offset", ctypes.c_size_t), ("rows", ctypes.c_size_t),
                ("cols", ctypes.c_size_t), ("scale", ctypes.c_double)]


_bound = None


def _lib():
    global _bound
    if _bound is None:
        L = lib()
        i32, vp, sz, f64 = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_double
        P = ctypes.POINTER
        sig = {
            "ddl_linear_workspace": [i32, sz, sz, sz, P(sz)],
            "ddl_linear": [P(ddl_linear_args), vp, sz, vp],
            "ddl_linear_dgrad": [P(ddl_dgrad_args), vp, sz, vp],
            "ddl_linear_wgrad": [P(ddl_wgrad_args), vp, sz, vp],
            "ddl_adamw_create": [P(vp), P(sz), P(sz), i32],
            "ddl_adamw_step": [vp, vp, i32, vp, vp, P(vp), i32, vp, i32, f64, f64, f64, f64, f64,
                               ctypes.c_longlong, vp],
            "ddl_adamw_destroy": [vp],
            "ddl_muon_create": [P(vp), P(ddl_muon_matrix), i32],
            "ddl_muon_orthogonalise": [vp, vp, vp, i32, vp],
            "ddl_muon_step": [vp, vp, i32, vp, P(vp), i32, vp, i32, f64, f64, i32, f64, vp],
            "ddl_muon_destroy": [vp],
        }
        for name, args in sig.items():
            fn = getattr(L, name)
            fn.argtypes, fn.restype = args, i32
        _bound = L
    return _bound


def _type(t, what):
    code = _TYPES.get(str(t.dtype))
    if code is None:
        raise ValueError(f"{what} has type {t.dtype}: expected float32, float16 or bfloat16")
    return code


def _act(act):
    if act not in ACTS:
        raise ValueError(f"unknown activation {act!r}: expected one of {', '.join(ACTS)}")
    return ACTS[act]


def _matrix(t, shape, like, what):
    """(pointer, row stride) of a 2-D tensor whose rows are contiguous."""
    if t is None:
        return None, 0
    if len(t.shape) != 2 or (shape is not None and tuple(t.shape) != tuple(shape)):
        raise ValueError(f"{what} has shape {tuple(t.shape)}: expected {shape}")
    if not t.is_cuda or (like is not None and t.device != like.device):
        raise ValueError(f"{what} is on {t.device}: expected a GPU tensor"
                         + (f" on {like.device}" if like is not None else ""))
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{what}'s rows are not contiguous (strides {tuple(t.stride())})")
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{what}'s rows overlap (strides {tuple(t.stride())})")
    return t.data_ptr(), t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _vector(t, n, like, what):
    if t is None:
        return None
    if tuple(t.shape) != (n,) or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{what} has shape {tuple(t.shape)}, strides {tuple(t.stride())}: "
                         f"expected {n} contiguous elements")
    if not t.is_cuda or t.device != like.device:
        raise ValueError(f"{what} is on {t.device}: expected {like.device}")
    return t.data_ptr()


def _same_type(like, **tensors):
    for name, t in tensors.items():
        if t is not None and t.dtype != like.dtype:
            raise ValueError(f"{name} has type {t.dtype}: expected {like.dtype}")


def _workspace(ws, like):
    if ws is None:
        return None, 0
    if not ws.is_cuda or ws.device != like.device or not ws.is_contiguous():
        raise ValueError(f"workspace: expected contiguous memory on {like.device}")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def linear_workspace(op, m, n, k):
    """Bytes of workspace that `op` ("forward", "dgrad" or "wgrad") takes for
    x m x k and w n x k (ddl_linear_workspace); may be 0."""
    if op not in _LINEAR_OPS:
        raise ValueError(f"unknown operation {op!r}: expected one of {', '.join(_LINEAR_OPS)}")
    if min(m, n, k) < 0:
        raise ValueError(f"negative size in ({m}, {n}, {k})")
    b = ctypes.c_size_t()
    _check(_lib().ddl_linear_workspace(_LINEAR_OPS[op], m, n, k, ctypes.byref(b)),
           "ddl_linear_workspace")
    return b.value


def linear(x, w, y, bias=None, act="none", residual=None, z=None, workspace=None, stream=None):
    """y = act(x w^T + bias) + residual into y; the activation's argument into
    z, where given (ddl_linear).  x (m, k), w (n, k), y, residual and z (m, n),
    bias (n), all float16 or all bfloat16."""
    a = ddl_linear_args()
    a.x, a.ldx = _matrix(x, None, None, "x")
    a.m, a.k = x.shape
    a.w, a.ldw = _matrix(w, (w.shape[0], a.k), x, "w")
    a.n = w.shape[0]
    a.dtype, a.act = _type(x, "x"), _act(act)
    _same_type(x, w=w, y=y, bias=bias, residual=residual, z=z)
    a.y, a.ldy = _matrix(y, (a.m, a.n), x, "y")
    a.bias = _vector(bias, a.n, x, "bias")
    a.residual, a.ldr = _matrix(residual, (a.m, a.n), x, "residual")
    a.z, a.ldz = _matrix(z, (a.m, a.n), x, "z")
    ws, size = _workspace(workspace, x)
    _check(_lib().ddl_linear(ctypes.byref(a), ws, size, _ptr(stream)), "ddl_linear")


def linear_dgrad(dz, w, dx, residual=None, act="none", z_prev=None, dz_prev=None, workspace=None,
                 stream=None):
    """dx = dz w + residual into dx and, where z_prev is given, dx act'(z_prev)
    into dz_prev: the gradient of the layer before, whose activation is act
    (ddl_linear_dgrad).  dz (m, n), w (n, k), the others (m, k)."""
    a = ddl_dgrad_args()
    a.dz, a.lddz = _matrix(dz, None, None, "dz")
    a.m, a.n = dz.shape
    a.w, a.ldw = _matrix(w, (a.n, w.shape[-1]), dz, "w")
    a.k = w.shape[1]
    a.dtype, a.act = _type(dz, "dz"), _act(act)
    if (z_prev is None) != (dz_prev is None) or (z_prev is None and act != "none"):
        raise ValueError("z_prev and dz_prev go together, and with an activation")
    _same_type(dz, w=w, dx=dx, residual=residual, z_prev=z_prev, dz_prev=dz_prev)
    a.dx, a.lddx = _matrix(dx, (a.m, a.k), dz, "dx")
    a.residual, a.ldr = _matrix(residual, (a.m, a.k), dz, "residual")
    a.z_prev, a.ldz_prev = _matrix(z_prev, (a.m, a.k), dz, "z_prev")
    a.dz_prev, a.lddz_prev = _matrix(dz_prev, (a.m, a.k), dz, "dz_prev")
    ws, size = _workspace(workspace, dz)
    _check(_lib().ddl_linear_dgrad(ctypes.byref(a), ws, size, _ptr(stream)), "ddl_linear_dgrad")


def linear_wgrad(dz, x, dw, db=None, accumulate=False, workspace=None, stream=None):
    """dw = dz^T x and db = dz's column sums, or added to them (ddl_linear_wgrad).
    dz (m, n), x (m, k); dw (n, k) and db (n) in float32 or in dz's type."""
    a = ddl_wgrad_args()
    a.dz, a.lddz = _matrix(dz, None, None, "dz")
    a.m, a.n = dz.shape
    a.x, a.ldx = _matrix(x, (a.m, x.shape[-1]), dz, "x")
    a.k = x.shape[1]
    a.dtype, a.out_dtype, a.accumulate = _type(dz, "dz"), _type(dw, "dw"), int(bool(accumulate))
    _same_type(dz, x=x)
    _same_type(dw, db=db)
    a.dw, a.lddw = _matrix(dw, (a.n, a.k), dz, "dw")
    a.db = _vector(db, a.n, dz, "db")
    ws, size = _workspace(workspace, dz)
    _check(_lib().ddl_linear_wgrad(ctypes.byref(a), ws, size, _ptr(stream)), "ddl_linear_wgrad")


def _flat(t, need, what, types=None, like=None):
    """The pointer of a flat buffer of at least `need` elements."""
    if t is None:
        return None
    if not t.is_cuda or (like is not None and t.device != like.device):
        raise ValueError(f"{what} is on {t.device}: expected a GPU tensor"
                         + (f" on {like.device}" if like is not None else ""))
    if not t.is_contiguous() or t.numel() < need:
        raise ValueError(f"{what} has {t.numel()} elements, strides {tuple(t.stride())}: "
                         f"expected at least {need}, contiguous")
    if types is not None and str(t.dtype) not in types:
        raise ValueError(f"{what} has type {t.dtype}: expected {' or '.join(types)}")
    return t.data_ptr()


_F32 = ("torch.float32",)
_F16S = ("torch.float16", "torch.bfloat16")


def _weights(weights, need, like):
    if not weights:
        raise ValueError("expected at least one replica of the weights")
    return (ctypes.c_void_p * len(weights))(
        *[_flat(w, need, f"weights[{i}]", _F32, like) for i, w in enumerate(weights)])


class _Optimizer:
    _destroy = None
    handle = None

    def destroy(self):
        if self.handle:
            h, self.handle = self.handle, None
            _check(getattr(_lib(), self._destroy)(h), self._destroy)

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


class AdamW(_Optimizer):
    """AdamW over spans [(offset, count)] of flat buffers (ddl_adamw_*)."""
    _destroy = "ddl_adamw_destroy"

    def __init__(self, spans):
        spans = [(int(o), int(c)) for o, c in spans]
        if any(o < 0 or c < 0 for o, c in spans):
            raise ValueError("negative offset or count")
        n = len(spans)
        offs = (ctypes.c_size_t * max(1, n))(*[o for o, _ in spans])
        cnts = (ctypes.c_size_t * max(1, n))(*[c for _, c in spans])
        self.need = max([o + c for o, c in spans if c], default=0)
        h = ctypes.c_void_p()
        _check(_lib().ddl_adamw_create(ctypes.byref(h), offs, cnts, n), "ddl_adamw_create")
        self.handle = h

    def step(self, grad, m, v, weights, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0,
             step=1, copy=None, stream=None):
        """One step on every replica in `weights`; `step` counts from 1; copy: a
        16-bit buffer that receives the new weights, or None."""
        n = self.need
        _check(_lib().ddl_adamw_step(
            self.handle, _flat(grad, n, "grad"), _type(grad, "grad"),
            _flat(m, n, "m", _F32, grad), _flat(v, n, "v", _F32, grad),
            _weights(weights, n, grad), len(weights), _flat(copy, n, "copy", _F16S, grad),
            _type(copy, "copy") if copy is not None else 0, float(lr), float(beta1),
            float(beta2), float(eps), float(weight_decay), int(step), _ptr(stream)),
            "ddl_adamw_step")


class Muon(_Optimizer):
    """Muon over matrices [(offset, rows, cols, scale)] of flat buffers
    (ddl_muon_*); scale multiplies the matrix's update."""
    _destroy = "ddl_muon_destroy"

    def __init__(self, matrices):
        matrices = [(int(o), int(r), int(c), float(s)) for o, r, c, s in matrices]
        if any(min(o, r, c) < 0 for o, r, c, _ in matrices):
            raise ValueError("negative offset, rows or cols")
        n = len(matrices)
        arr = (ddl_muon_matrix * max(1, n))()
        for i, (o, r, c, s) in enumerate(matrices):
            arr[i].offset, arr[i].rows, arr[i].cols, arr[i].scale = o, r, c, s
        self.need = max([o + r * c for o, r, c, _ in matrices if r * c], default=0)
        h = ctypes.c_void_p()
        _check(_lib().ddl_muon_create(ctypes.byref(h), arr, n), "ddl_muon_create")
        self.handle = h

    def orthogonalise(self, grad, out, stream=None):
        """out = the nearly orthogonal form of every matrix of grad (same type)."""
        _same_type(grad, out=out)
        _check(_lib().ddl_muon_orthogonalise(
            self.handle, _flat(grad, self.need, "grad"), _flat(out, self.need, "out", None, grad),
            _type(grad, "grad"), _ptr(stream)), "ddl_muon_orthogonalise")

    def step(self, grad, momentum, weights, lr, momentum_decay=0.95, nesterov=True,
             weight_decay=0.0, copy=None, stream=None):
        """momentum = momentum_decay momentum + grad, then the orthogonalised
        update of every replica in `weights` (see ddl_muon_step)."""
        n = self.need
        _check(_lib().ddl_muon_step(
            self.handle, _flat(grad, n, "grad"), _type(grad, "grad"),
            _flat(momentum, n, "momentum", _F32, grad), _weights(weights, n, grad), len(weights),
            _flat(copy, n, "copy", _F16S, grad), _type(copy, "copy") if copy is not None else 0,
            float(lr), float(momentum_decay), int(bool(nesterov)), float(weight_decay),
            _ptr(stream)), "ddl_muon_step")
