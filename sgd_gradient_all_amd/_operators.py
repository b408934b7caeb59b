"""The linear layer's products and the Muon and AdamW steps (include/ddl.h).

Argument checks and marshalling only.  Arrays are torch tensors (or objects
like them) on the current GPU; streams as elsewhere (None = the null stream).
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


# The checks below run before every call, and a decoded token's product is done
# in a few microseconds: types are looked up by object, devices by index.
_type_codes = {}


def _type(t, what):
    code = _type_codes.get(t.dtype)
    if code is None:
        code = _TYPES.get(str(t.dtype))
        if code is None:
            raise ValueError(f"{what} has type {t.dtype}: expected float32, float16 or bfloat16")
        _type_codes[t.dtype] = code
    return code


def _act(act):
    code = ACTS.get(act)
    if code is None:
        raise ValueError(f"unknown activation {act!r}: expected one of {', '.join(ACTS)}")
    return code


_get_device = None


def _current_device():
    """The index of the GPU that kernels are launched on."""
    global _get_device
    if _get_device is None:
        _get_device = _lib().hipGetDevice
    now = ctypes.c_int()
    if _get_device(ctypes.byref(now)):
        raise RuntimeError("no current GPU")
    return now.value


def _device(t, what):
    """The index of the GPU that t is on, which has to be the current one."""
    d = t.get_device()
    if d < 0:
        raise ValueError(f"{what} is on {t.device}: expected a GPU tensor")
    now = _current_device()
    if d != now:
        raise ValueError(f"{what} is on {t.device}: expected a tensor of the current GPU, {now}")
    return d


def _matrix(t, rows, cols, device, dtype, what):
    """(pointer, row stride) of a rows x cols tensor whose rows are contiguous."""
    if t is None:
        return None, 0
    shape = t.shape
    if len(shape) != 2 or shape[0] != rows or shape[1] != cols:
        raise ValueError(f"{what} has shape {tuple(shape)}: expected ({rows}, {cols})")
    if t.get_device() != device:
        raise ValueError(f"{what} is on {t.device}: expected a GPU tensor on device {device}")
    if t.dtype != dtype:
        raise ValueError(f"{what} has type {t.dtype}: expected {dtype}")
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{what}'s rows are not contiguous (strides {t.stride()})")
    if rows <= 1:
        return t.data_ptr(), cols
    if ld < cols:
        raise ValueError(f"{what}'s rows overlap (strides {t.stride()})")
    return t.data_ptr(), ld


def _two(t, what):
    if len(t.shape) != 2:
        raise ValueError(f"{what} has shape {tuple(t.shape)}: expected two dimensions")
    return t.shape


def _vector(t, n, device, dtype, what):
    if t is None:
        return None
    if len(t.shape) != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{what} has shape {tuple(t.shape)}, strides {tuple(t.stride())}: "
                         f"expected {n} contiguous elements")
    if t.get_device() != device or t.dtype != dtype:
        raise ValueError(f"{what} is {t.dtype} on {t.device}: expected {dtype} on device {device}")
    return t.data_ptr()


def _workspace(ws, device):
    if ws is None:
        return None, 0
    if ws.get_device() != device or not ws.is_contiguous():
        raise ValueError(f"workspace: expected contiguous memory on device {device}")
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
    m, k = _two(x, "x")
    n = _two(w, "w")[0]
    code, act = _type(x, "x"), _act(act)
    d, t = _device(x, "x"), x.dtype
    px, ldx = _matrix(x, m, k, d, t, "x")
    pw, ldw = _matrix(w, n, k, d, t, "w")
    py, ldy = _matrix(y, m, n, d, t, "y")
    pr, ldr = _matrix(residual, m, n, d, t, "residual")
    pz, ldz = _matrix(z, m, n, d, t, "z")
    a = ddl_linear_args(m, n, k, code, act, px, ldx, pw, ldw, _vector(bias, n, d, t, "bias"), pr,
                        ldr, py, ldy, pz, ldz)
    ws, size = _workspace(workspace, d)
    rc = (_bound or _lib()).ddl_linear(ctypes.byref(a), ws, size, _ptr(stream))
    if rc:
        _check(rc, "ddl_linear")


def linear_dgrad(dz, w, dx, residual=None, act="none", z_prev=None, dz_prev=None, workspace=None,
                 stream=None):
    """dx = dz w + residual into dx and, where z_prev is given, dx act'(z_prev)
    into dz_prev: the gradient of the layer before, whose activation is act
    (ddl_linear_dgrad).  dz (m, n), w (n, k), the others (m, k)."""
    m, n = _two(dz, "dz")
    k = _two(w, "w")[1]
    code, act_code = _type(dz, "dz"), _act(act)
    if (z_prev is None) != (dz_prev is None) or (z_prev is None and act != "none"):
        raise ValueError("z_prev and dz_prev go together, and with an activation")
    d, t = _device(dz, "dz"), dz.dtype
    pz, ldz = _matrix(dz, m, n, d, t, "dz")
    pw, ldw = _matrix(w, n, k, d, t, "w")
    px, ldx = _matrix(dx, m, k, d, t, "dx")
    pr, ldr = _matrix(residual, m, k, d, t, "residual")
    pzp, ldzp = _matrix(z_prev, m, k, d, t, "z_prev")
    pdzp, lddzp = _matrix(dz_prev, m, k, d, t, "dz_prev")
    a = ddl_dgrad_args(m, n, k, code, act_code, pz, ldz, pw, ldw, pr, ldr, px, ldx, pzp, ldzp,
                       pdzp, lddzp)
    ws, size = _workspace(workspace, d)
    rc = (_bound or _lib()).ddl_linear_dgrad(ctypes.byref(a), ws, size, _ptr(stream))
    if rc:
        _check(rc, "ddl_linear_dgrad")


def linear_wgrad(dz, x, dw, db=None, accumulate=False, workspace=None, stream=None):
    """dw = dz^T x and db = dz's column sums, or added to them (ddl_linear_wgrad).
    dz (m, n), x (m, k); dw (n, k) and db (n) in float32 or in dz's type."""
    m, n = _two(dz, "dz")
    k = _two(x, "x")[1]
    code, out = _type(dz, "dz"), _type(dw, "dw")
    d, t = _device(dz, "dz"), dz.dtype
    pz, ldz = _matrix(dz, m, n, d, t, "dz")
    px, ldx = _matrix(x, m, k, d, t, "x")
    pw, ldw = _matrix(dw, n, k, d, dw.dtype, "dw")
    a = ddl_wgrad_args(m, n, k, code, out, int(bool(accumulate)), pz, ldz, px, ldx, pw, ldw,
                       _vector(db, n, d, dw.dtype, "db"))
    ws, size = _workspace(workspace, d)
    rc = (_bound or _lib()).ddl_linear_wgrad(ctypes.byref(a), ws, size, _ptr(stream))
    if rc:
        _check(rc, "ddl_linear_wgrad")


def _flat(t, need, what, codes=None, device=None):
    """The pointer of a flat buffer of at least `need` elements."""
    if t is None:
        return None
    if device is None:
        _device(t, what)
    elif t.get_device() != device:
        raise ValueError(f"{what} is on {t.device}: expected a GPU tensor on device {device}")
    if not t.is_contiguous() or t.numel() < need:
        raise ValueError(f"{what} has {t.numel()} elements, strides {tuple(t.stride())}: "
                         f"expected at least {need}, contiguous")
    if codes is not None and _type(t, what) not in codes:
        raise ValueError(f"{what} has type {t.dtype}, which this argument does not take")
    return t.data_ptr()


_F32 = (DDL_F32,)
_F16S = (DDL_F16, DDL_BF16)


def _weights(weights, need, device):
    if not weights:
        raise ValueError("expected at least one replica of the weights")
    return (ctypes.c_void_p * len(weights))(
        *[_flat(w, need, "weights", _F32, device) for w in weights])


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
        n, d = self.need, _device(grad, "grad")
        rc = _lib().ddl_adamw_step(
            self.handle, _flat(grad, n, "grad", None, d), _type(grad, "grad"),
            _flat(m, n, "m", _F32, d), _flat(v, n, "v", _F32, d), _weights(weights, n, d),
            len(weights), _flat(copy, n, "copy", _F16S, d),
            _type(copy, "copy") if copy is not None else 0, lr, beta1, beta2, eps, weight_decay,
            step, _ptr(stream))
        if rc:
            _check(rc, "ddl_adamw_step")


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
        if grad.dtype != out.dtype:
            raise ValueError(f"out has type {out.dtype}: expected {grad.dtype}")
        d = _device(grad, "grad")
        rc = _lib().ddl_muon_orthogonalise(
            self.handle, _flat(grad, self.need, "grad", None, d),
            _flat(out, self.need, "out", None, d), _type(grad, "grad"), _ptr(stream))
        if rc:
            _check(rc, "ddl_muon_orthogonalise")

    def step(self, grad, momentum, weights, lr, momentum_decay=0.95, nesterov=True,
             weight_decay=0.0, copy=None, stream=None):
        """momentum = momentum_decay momentum + grad, then the orthogonalised
        update of every replica in `weights` (see ddl_muon_step)."""
        n, d = self.need, _device(grad, "grad")
        rc = _lib().ddl_muon_step(
            self.handle, _flat(grad, n, "grad", None, d), _type(grad, "grad"),
            _flat(momentum, n, "momentum", _F32, d), _weights(weights, n, d), len(weights),
            _flat(copy, n, "copy", _F16S, d), _type(copy, "copy") if copy is not None else 0, lr,
            momentum_decay, int(bool(nesterov)), weight_decay, _ptr(stream))
        if rc:
            _check(rc, "ddl_muon_step")
