"""Training of the experts and of the norm in front of them, on one GPU.

``TrainableExperts`` strings libmoe's training operators together over the
rows of a dispatch: gate/up product, SwiGLU, down product, and their
gradients.  ``LayerNorm`` is the norm before the layer.  As in ``layer``,
torch provides device memory and streams only.

A step of the layer's training is made of

    x = norm.forward(u)                      # the layer's input
    L.moe_route(...); L.moe_dispatch(...)    # idx, w, offsets, perm, inv
    y = experts.forward(x_rows, offsets)     # x_rows = x[perm // top_k]
    L.moe_combine(...)
    ...
    dx_rows = experts.backward(dy)           # dy = w * dh of each row
    du = norm.backward(dx)                   # dx = sums of dx_rows by token
    m = beta * m + experts.dW13              # the optimiser's momentum
    update = orthogonalize(m)

Each call runs on ``stream`` (a torch stream or a raw handle; None: the current
one), and so does every allocation that it makes, its results among them.  What
it reads and writes beside them is recorded on a ``stream`` that is not the
current one: the memory of an input that the caller lets go of is given to no
other before the call is done with it.  (A raw handle has to outlive the tensors
passed with it.  On the current stream torch's own rule holds: a tensor made on
another one is the caller's to record.)
"""
from __future__ import annotations

import contextlib

import torch

from . import _lib as L

_DTYPE = {torch.bfloat16: L.MOE_DTYPE_BF16, torch.float32: L.MOE_DTYPE_F32}


def _on_current(t, what):
    # the library launches on the current device
    if not t.is_cuda or t.device.index != torch.cuda.current_device():
        raise ValueError(f"{what} has to be on the current CUDA device, not on {t.device}")
    return t


def _torch_stream(stream):
    """The torch stream of a raw handle.  0 and 1 are the default stream's (for
    0 ExternalStream makes a new one)."""
    if not isinstance(stream, int):
        return stream
    return torch.cuda.ExternalStream(stream) if stream > 1 else torch.cuda.default_stream()


def _on(stream):
    """A context in which torch allocates for ``stream``."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(_torch_stream(stream))


def _record(stream, *tensors):
    """The tensors' memory is in use until ``stream`` has done what it was given
    by the time that they are let go of."""
    if stream is None or L._stream(stream) == L._stream(None):
        return  # 1 us a tensor, a step of 64 rows 112 us for 87
    stream = _torch_stream(stream)
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def _same_stream(saved, stream):
    # the saved tensors return to their stream's pool with the backward pass
    if L._stream(stream) != saved:
        raise ValueError("backward() on another stream than its forward()")


def _scratch(nbytes, device):
    # zeroed: a workspace starts with its status word
    return torch.zeros(max(256, nbytes), dtype=torch.uint8, device=device)


class TrainableExperts:
    """SwiGLU experts over ragged rows, with their weights' gradients.

    ``W13`` [n, 2*inter, d] is packed as by ``moe_pack_w13``, ``W2`` is
    [n, d, inter].  ``dW13`` and ``dW2`` are float32, accumulated over the
    ``backward`` calls since ``zero_grad``.  Rows that no expert owns (behind the
    last offset of a padded batch) reach none of them; in the results they hold
    anything."""

    def __init__(self, W13: torch.Tensor, W2: torch.Tensor):
        n, two_inter, d = W13.shape
        if (two_inter % 128 != 0 or W2.shape != (n, d, two_inter // 2) or W2.dtype != W13.dtype
                or W13.dtype not in _DTYPE or W2.device != W13.device
                or not W13.is_contiguous() or not W2.is_contiguous()):
            raise ValueError("W13 [n, 2*inter, d] and W2 [n, d, inter] have to be contiguous, of "
                             "one float dtype and device, inter a multiple of 64")
        self.W13, self.W2 = W13, W2
        self.n, self.inter, self.d = n, two_inter // 2, d
        self.dtype = W13.dtype
        self.dW13 = torch.empty(W13.shape, dtype=torch.float32, device=W13.device)
        self.dW2 = torch.empty(W2.shape, dtype=torch.float32, device=W2.device)
        self.ws = _scratch(256, W13.device)
        self._saved = None
        self._have_grad = False
        self._last = None  # raw stream of the last call

    def _shape(self, rows, n, k, flags=0):
        return L.make_grouped_shape(rows, self.n, n, k, _DTYPE[self.dtype], flags)

    def _rows(self, t, width, what):
        if t.dim() != 2 or t.shape[1] != width or t.dtype != self.dtype or not t.is_contiguous() \
                or t.device != self.W13.device:
            raise ValueError(f"{what} has to be contiguous [rows, {width}] of {self.dtype} beside "
                             "the weights")
        return _on_current(t, what)

    def forward(self, x: torch.Tensor, offsets: torch.Tensor, stream=None) -> torch.Tensor:
        """y[r] = FFN_g(x[r]) for the rows r of each expert g, which ``offsets``
        (int32 [n + 1], of ``moe_dispatch``) gives.  Keeps what ``backward``
        needs: x and offsets themselves, which must not change before it, on
        the same stream."""
        self._rows(x, self.d, "x")
        if offsets.dtype != torch.int32 or offsets.shape != (self.n + 1,) \
                or offsets.device != x.device or not offsets.is_contiguous():
            raise ValueError(f"offsets has to be contiguous int32 [{self.n + 1}] beside the weights")
        rows = x.shape[0]
        with _on(stream):
            gu, a = x.new_empty(rows, 2 * self.inter), x.new_empty(rows, self.inter)
            y = torch.empty_like(x)
        _record(stream, x, offsets, self.W13, self.W2, self.ws)
        self._last = L._stream(stream)
        L.moe_grouped_matmul(self._shape(rows, 2 * self.inter, self.d), x, offsets, self.W13, gu,
                             self.ws, stream=stream)
        L.moe_swiglu(L.make_swiglu_shape(rows, self.inter, _DTYPE[self.dtype]), gu, a, stream=stream)
        L.moe_grouped_matmul(self._shape(rows, self.d, self.inter), a, offsets, self.W2, y, self.ws,
                             stream=stream)
        self._saved = (x, offsets, gu, a, self._last)
        return y

    def backward(self, dy: torch.Tensor, stream=None) -> torch.Tensor:
        """The gradient of ``forward``'s x from that of its y; adds to dW13 and
        dW2.  Once per forward.  A refusal or a lack of memory leaves the
        forward and the gradients as they are; an error after dW2 was issued
        leaves the two apart, and the next call asks for ``zero_grad``."""
        if self._saved is None:
            raise RuntimeError("backward() without a forward() before it")
        x, offsets, gu, a, saved_on = self._saved
        if self._rows(dy, self.d, "dy").shape != x.shape:
            raise ValueError("dy has to have as many rows as x")
        _same_stream(saved_on, stream)
        if self._have_grad is None:
            raise RuntimeError("an earlier backward() failed between dW2 and dW13: zero_grad() first")
        rows, flags = x.shape[0], L.MOE_GROUPED_DW_F32
        if self._have_grad:
            flags |= L.MOE_GROUPED_DW_ACCUMULATE
        up = self._shape(rows, 2 * self.inter, self.d, flags)
        down = self._shape(rows, self.d, self.inter, flags)
        with _on(stream):
            da, dx = torch.empty_like(a), torch.empty_like(x)
        # up to here an error changes nothing
        self._saved = None
        _record(stream, dy, self.dW13, self.dW2)
        L.moe_grouped_matmul_dx(down, dy, offsets, self.W2, da, self.ws, stream=stream)
        L.moe_grouped_matmul_dw(down, dy, a, offsets, self.dW2, self.ws, stream=stream)
        self._have_grad = None  # until dW13 has what dW2 has
        # the pre-activations' gradient takes their place
        L.moe_swiglu_backward(L.make_swiglu_shape(rows, self.inter, _DTYPE[self.dtype]), gu, da, gu,
                              stream=stream)
        L.moe_grouped_matmul_dx(up, gu, offsets, self.W13, dx, self.ws, stream=stream)
        L.moe_grouped_matmul_dw(up, gu, x, offsets, self.dW13, self.ws, stream=stream)
        self._have_grad = True
        return dx

    def zero_grad(self):
        """The next ``backward`` overwrites dW13 and dW2."""
        self._have_grad = False

    def status(self, stream=None) -> int:
        """MOE_OK, or MOE_ERR_DEVICE_CHECK if a wait of a call before ran out;
        clears it.  Waits for ``stream`` (None: that of the last forward or
        backward, and the current one; replays of captured calls on another
        stream need it named)."""
        if stream is None and self._last not in (None, L._stream(None)):
            _torch_stream(self._last).synchronize()
        return L.moe_read_status(self.ws, stream=stream)


class LayerNorm:
    """Layer norm over the last axis of [T, d] rows, float32 weight and bias."""

    def __init__(self, gamma: torch.Tensor, beta: torch.Tensor | None = None, eps: float = 1e-5):
        for t in (gamma, beta):
            if t is not None and (t.dtype != torch.float32 or t.shape != gamma.shape
                                  or t.dim() != 1 or not t.is_contiguous()
                                  or t.device != gamma.device):
                raise ValueError("gamma and beta have to be contiguous float32 [d]")
        self.gamma, self.beta, self.eps = gamma, beta, eps
        self.dgamma = torch.empty_like(gamma)
        self.dbeta = None if beta is None else torch.empty_like(beta)
        self._saved = None
        self._have_grad = False

    def _shape(self, x):
        if x.dim() != 2 or x.shape[1] != self.gamma.shape[0] or x.dtype not in _DTYPE \
                or not x.is_contiguous() or x.device != self.gamma.device:
            raise ValueError(f"rows have to be contiguous [T, {self.gamma.shape[0]}], bfloat16 or "
                             "float32, beside gamma")
        _on_current(x, "x")
        return L.make_norm_shape(x.shape[0], x.shape[1], _DTYPE[x.dtype], self.eps)

    def forward(self, x: torch.Tensor, stream=None) -> torch.Tensor:
        """Keeps x itself, which must not change before ``backward``, on the
        same stream."""
        shape = self._shape(x)
        with _on(stream):
            y = torch.empty_like(x)
            mean = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
            rstd = torch.empty_like(mean)
        _record(stream, x, self.gamma, self.beta)
        L.moe_layer_norm(shape, x, self.gamma, self.beta, y, mean, rstd, stream=stream)
        self._saved = (x, mean, rstd, L._stream(stream))
        return y

    def backward(self, dy: torch.Tensor, stream=None, accumulate: bool = False) -> torch.Tensor:
        """The gradient of ``forward``'s x; writes dgamma and dbeta, or adds to
        what the ``backward`` calls since ``zero_grad`` left there (which
        ``TrainableExperts.backward`` always does)."""
        if self._saved is None:
            raise RuntimeError("backward() without a forward() before it")
        x, mean, rstd, saved_on = self._saved
        shape = self._shape(dy)
        if dy.shape != x.shape or dy.dtype != x.dtype:
            raise ValueError("dy has to be like x")
        _same_stream(saved_on, stream)
        dgamma, dbeta = self.dgamma, self.dbeta
        add = accumulate and self._have_grad
        with _on(stream):
            dx = torch.empty_like(x)
            # a workspace per call: captured ones may replay side by side
            ws = x.new_empty(max(256, L.moe_layer_norm_workspace_size(shape)), dtype=torch.uint8)
            if add:
                dgamma = torch.empty_like(dgamma)
                dbeta = None if dbeta is None else torch.empty_like(dbeta)
        self._saved = None  # up to here an error changes nothing
        _record(stream, dy, self.dgamma, self.dbeta)
        L.moe_layer_norm_backward(shape, dy, x, self.gamma, mean, rstd, dx, dgamma, dbeta, ws,
                                  stream=stream)
        if add:
            with _on(stream):
                self.dgamma += dgamma
                if dbeta is not None:
                    self.dbeta += dbeta
        self._have_grad = True
        return dx

    def zero_grad(self):
        """The next ``backward`` overwrites dgamma and dbeta."""
        self._have_grad = False


def _ortho_shape(m, steps):
    if m.dim() != 3 or m.dtype not in _DTYPE or not m.is_contiguous():
        raise ValueError("m has to be contiguous [n, rows, cols], bfloat16 or float32")
    _on_current(m, "m")
    return L.make_ortho_shape(*m.shape, steps, _DTYPE[m.dtype])


def orthogonalize_workspace(m: torch.Tensor, steps: int = 5, stream=None) -> torch.Tensor:
    """A workspace for ``orthogonalize`` of matrices like m, its status word
    zeroed on ``stream``.  One can serve call after call on a stream, and
    ``_lib.moe_read_status(ws, stream=stream)`` tells whether a wait of theirs
    ran out."""
    nbytes = max(256, L.moe_orthogonalize_workspace_size(_ortho_shape(m, steps)))
    with _on(stream):
        ws = torch.empty(nbytes, dtype=torch.uint8, device=m.device)
        ws[:4].zero_()
    return ws


def orthogonalize(m: torch.Tensor, steps: int = 5, coef=None, ws: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """Newton-Schulz orthogonalisation of each matrix of m [n, rows, cols], as
    bfloat16.  Of packed W13 matrices it is that of W1 on top of W3: the
    packing permutes rows, which the iteration commutes with.

    Without ``ws`` the call takes its own, whose status nobody can read: pass
    one of ``orthogonalize_workspace`` to learn of a wait that ran out."""
    shape = _ortho_shape(m, steps)
    # the library writes ws_bytes from its first one on
    if ws is not None and (ws.device != m.device or not ws.is_contiguous()):
        raise ValueError("ws has to be contiguous, on the device of m")
    with _on(stream):
        if ws is None:
            nbytes = max(256, L.moe_orthogonalize_workspace_size(shape))
            ws = torch.empty(nbytes, dtype=torch.uint8, device=m.device)
        o = torch.empty(m.shape, dtype=torch.bfloat16, device=m.device)
    _record(stream, m, ws)
    L.moe_orthogonalize(shape, m, o, ws, coef=coef, stream=stream)
    return o
