"""Layers over a frozen bf16 LM head that do not write the [M, V] logits: log-probabilities of
given tokens with entropy and top alternatives, and distillation from a teacher's top logits,
each with its gradient in the hidden states.  (A forward with ``save=True`` keeps their exponentials
in bf16 for the backward.)"""
from __future__ import annotations

import dataclasses
import threading
from ctypes import byref

import torch

from . import binding as _b

# The layers call the library without the binding's wrappers and torch.cuda.current_stream():
# a call on a small head takes the GPU about as long as these take the host.
_current_raw_stream = torch._C._cuda_getCurrentRawStream
_lib = _b.lib()


def _check(status: int, where: str):
    if status != _b.LORA_OK:
        raise _b.LoraError(status, where)


def _ptr(t):
    return None if t is None else t.data_ptr()


@dataclasses.dataclass
class TokenLogProbs:
    """What :meth:`LoraTokenLogProbs.forward` returns.  ``logprob`` has the shape of the ids
    given (None without ids); ``entropy`` [M]; ``lse`` [M]; ``top_ids`` int32 and
    ``top_logprob`` [M, k] (None for k = 0).  The other fields belong to the backward."""

    logprob: torch.Tensor | None
    lse: torch.Tensor
    entropy: torch.Tensor | None
    top_ids: torch.Tensor | None = None
    top_logprob: torch.Tensor | None = None
    saved: torch.Tensor | None = None
    tokens: int = 0
    stream: int = 0         # the stream that saved was taken on
    capture: int = 0        # the graph capture that the forward was part of, 0: none


@dataclasses.dataclass
class DistillLoss:
    """What :meth:`LoraDistill.forward` returns: ``loss`` [M], ``lse`` [M]; the other fields belong
    to the backward."""

    loss: torch.Tensor
    lse: torch.Tensor
    saved: torch.Tensor | None = None
    tokens: int = 0
    stream: int = 0         # the stream that saved was taken on
    capture: int = 0        # the graph capture that the forward was part of, 0: none


class _HeadLayer:
    """Checks, streams and workspaces shared by the head's layers.

    A call runs on ``stream`` (default: the current stream of X's device) and takes its outputs
    and its workspace from that stream's memory, one workspace a stream, so calls on two streams
    do not meet in it; a lock keeps two threads' calls on one stream apart.  A call under CUDA
    graph capture takes a workspace of its own from the graph's memory.  Tensors start on a 16-byte
    boundary (a slice such as ``ids[1:]`` may need a copy).
    """

    def __init__(self, W: "_b.LoraWeight", ignore_index: int = -100, temperature: float = 1.0, slice_: int = 0):
        if not float(temperature) > 0.0:
            raise ValueError("temperature must be positive")
        if W.fmt != _b.LORA_W_BF16:
            raise _b.LoraError(_b.LORA_ERR_UNSUPPORTED, "the LM head must be bf16")
        self.W, self.ignore_index, self.slice = W, int(ignore_index), int(slice_)
        self.scale = 1.0 / float(temperature)
        self._ws = {}
        self._sizes = {}
        self._lock = threading.Lock()

    def _run(self, call, X, stream, *tensors):
        """``call(handle)`` with X's device and ``stream`` current; returns what it returns.  The caller's
        tensors and the head keep their memory until a call on another stream has run."""
        index = X.device.index
        if stream is None and index == torch.cuda.current_device():
            with self._lock:
                return call(_current_raw_stream(index))  # the usual case, without the context managers
        with torch.cuda.device(index):
            if isinstance(stream, int):
                stream = torch.cuda.ExternalStream(stream, device=X.device)
            elif stream is None:
                stream = torch.cuda.current_stream()
            if stream != torch.cuda.current_stream():
                for t in (X, self.W.data, *tensors):
                    if t is not None:
                        t.record_stream(stream)
            with torch.cuda.stream(stream), self._lock:
                return call(stream.cuda_stream)

    def _bytes(self, fn, *sizes) -> int:
        """A workspace size, asked for once (it is a function of the sizes alone)."""
        n = self._sizes.get((fn, sizes))
        if n is None:
            if len(self._sizes) >= 4096:
                self._sizes.clear()
            n = self._sizes[(fn, sizes)] = fn(*sizes)
            if n == 0:
                raise _b.LoraError(_b.LORA_ERR_UNSUPPORTED, fn.__name__)
        return n

    def _workspace(self, nbytes: int, device, stream: int) -> torch.Tensor:
        """At least nbytes.  A call passes the library the size that it asked for, not the buffer's: the
        backward's slices go by it."""
        if torch.cuda.is_current_stream_capturing():
            ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
            ws[:256].zero_()
            return ws
        key = (device.index, stream)
        ws = self._ws.get(key)
        if ws is None or ws.numel() < nbytes:
            head = torch.zeros(256, dtype=torch.uint8, device=device) if ws is None else ws[:256]
            ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
            ws[:256].copy_(head)  # a larger one keeps the status
            self._ws[key] = ws
        return ws

    def status(self) -> int:
        """The first device status that is not LORA_OK of the calls made so far (synchronizes),
        calls under graph capture aside."""
        out = _b.LORA_OK
        with self._lock:  # another thread's call may add or replace a workspace
            for (dev, stream), ws in self._ws.items():
                with torch.cuda.device(dev):
                    st = _b.lora_device_status(ws, stream)
                out = st if out == _b.LORA_OK else out
        return out

    def _hidden(self, X):
        if not (isinstance(X, torch.Tensor) and X.is_cuda and X.dtype == torch.bfloat16 and X.dim() == 2
                and X.is_contiguous()):
            raise ValueError("X must be a contiguous bf16 CUDA tensor [M, D]")
        if X.shape[1] != self.W.K:
            raise ValueError(f"X has {X.shape[1]} columns, the head {self.W.K}")
        if X.device != self.W.data.device:
            raise ValueError(f"X is on {X.device}, the head on {self.W.data.device}")
        return X.shape[0]

    @staticmethod
    def _like(t, name, dtype, shape, device):
        if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.shape == shape and t.device == device
                and t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on {device}")
        return t

    def _ids(self, ids, M, device, flat):
        """Checks ids [M, n] (or [M], where ``flat`` allows it); returns n."""
        if not (isinstance(ids, torch.Tensor) and ids.dim() in ((1, 2) if flat else (2,)) and ids.shape[0] == M):
            raise ValueError(f"ids must be an int32 tensor [{M}, n]" + (f" or [{M}]" if flat else ""))
        n = ids.shape[1] if ids.dim() == 2 else 1
        if not 1 <= n <= _b.LORA_HEAD_MAX_IDS:
            raise ValueError(f"between 1 and {_b.LORA_HEAD_MAX_IDS} tokens a row")
        self._like(ids, "ids", torch.int32, ids.shape, device)
        return n

    @staticmethod
    def _own(fwd, cls):
        """Refuses the other operator's forward: the saved buffers are laid out differently (distillation's
        holds a map of its rows, which the backward follows)."""
        if not isinstance(fwd, cls):
            raise ValueError(f"fwd must be the {cls.__name__} of this operator's forward")

    def _slice(self, M):
        """Vocabulary rows a slice of a backward that recomputes: about 1 GiB of dz unless set."""
        if self.slice > 0:
            return self.slice
        return max(256, min(self.W.N, (1 << 30) // (2 * max(M, 1)) // 256 * 256))

    def _saved(self, M, n, device):
        return torch.empty(self._bytes(_b.head_saved_bytes, M, self.W.N, n), dtype=torch.uint8, device=device)

    def _saved_of(self, fwd, M, n, stream):
        """The forward's saved buffer for this backward, which overwrites it (None: recompute); _used
        drops it once the call has been made.  It serves a backward that runs once for each run of the
        forward: both ordinary calls, or both in one graph."""
        if fwd.saved is None or fwd.capture != self._capture(stream):
            return None
        saved = fwd.saved
        if fwd.tokens != n or saved.numel() != self._bytes(_b.head_saved_bytes, M, self.W.N, n):
            raise ValueError("the forward was saved with other sizes (rows, tokens a row or vocabulary)")
        if fwd.stream != stream:  # not handed out again before this backward has run
            saved.record_stream(torch.cuda.current_stream())
        return saved

    @staticmethod
    def _used(fwd, saved):
        if saved is not None:
            fwd.saved = None

    @staticmethod
    def _capture(stream):
        return _b.lora_stream_capture_id(stream) if torch.cuda.is_current_stream_capturing() else 0

    @classmethod
    def _mark(cls, out, stream):
        if out.saved is not None:
            out.stream, out.capture = stream, cls._capture(stream)
        return out

    def _bwd_bytes(self, M, n, saved) -> int:
        slice_ = 0 if saved is not None else self._slice(M)
        return self._bytes(_b.head_bwd_workspace_bytes, M, self.W.K, self.W.N, n, slice_)

    def _check_dX(self, dX, X):
        if dX is not None:
            self._like(dX, "dX", torch.bfloat16, X.shape, X.device)


class LoraTokenLogProbs(_HeadLayer):
    """Log-probabilities of given tokens under softmax(X·Wᵀ/temperature), with the entropy of
    each row and its ``top_k`` alternatives, over a frozen bf16 LM head ``W [V, D]`` (a
    :class:`LoraWeight`), without writing the ``[M, V]`` logits.

    ``forward(X, ids)``: X bf16 [M, D], ids int32 [M] or [M, n] (n <= 128, entries equal to
    ``ignore_index`` have logprob 0 and no gradient) or None; top_k <= 32 (its workspace, up to 1.25 GiB,
    stays with the layer, one a stream).  With ``save=True`` the
    forward keeps 2·M·V bytes for one backward, which then skips recomputing the logits (a later
    backward of the same forward, or one of which only either was captured into a graph, or each into
    its own, recomputes them, in vocabulary slices of ``slice_`` rows, by default as many as take 1 GiB).
    ``backward`` returns dX for upstream gradients of the log-probabilities (shape of ids) and of the
    entropies ([M]).
    """

    def forward(self, X: torch.Tensor, ids: torch.Tensor | None = None, top_k: int = 0, entropy: bool = True,
                save: bool = False, stream=None) -> TokenLogProbs:
        M, dev = self._hidden(X), X.device
        n = 0 if ids is None else self._ids(ids, M, dev, True)
        k = int(top_k)
        if not 0 <= k <= min(_b.LORA_HEAD_MAX_TOP, self.W.N):
            raise ValueError(f"top_k must be between 0 and {min(_b.LORA_HEAD_MAX_TOP, self.W.N)}")

        def call(handle):
            # empty_like and sizes as numbers: half of what empty() takes with a shape
            f32 = torch.float32
            lse = torch.empty(M, dtype=f32, device=dev)
            out = TokenLogProbs(
                None if ids is None else torch.empty_like(ids, dtype=f32),
                lse,
                torch.empty_like(lse) if entropy else None,
                torch.empty(M, k, dtype=torch.int32, device=dev) if k else None,
                torch.empty(M, k, dtype=f32, device=dev) if k else None,
                self._saved(M, n, dev) if save else None, n)
            size = self._bytes(_b.head_fwd_workspace_bytes, M, self.W.K, self.W.N, n, k)
            ws = self._workspace(size, dev, handle)
            _check(_lib.lora_logprob_fwd(X.data_ptr(), M, byref(self.W.c_struct()), _ptr(ids), n, self.ignore_index,
                                         self.scale, k, _ptr(out.logprob), _ptr(out.entropy), out.lse.data_ptr(),
                                         _ptr(out.top_ids), _ptr(out.top_logprob), _ptr(out.saved), ws.data_ptr(),
                                         size, handle), "lora_logprob_fwd")
            return self._mark(out, handle)

        return self._run(call, X, stream, ids)

    def backward(self, X: torch.Tensor, ids: torch.Tensor | None, fwd: TokenLogProbs,
                 dlogprob: torch.Tensor | None = None, dentropy: torch.Tensor | None = None, dX=None,
                 stream=None) -> torch.Tensor:
        M, dev = self._hidden(X), X.device
        n = 0 if ids is None else self._ids(ids, M, dev, True)
        self._own(fwd, TokenLogProbs)
        if dlogprob is not None:
            if ids is None:
                raise ValueError("dlogprob without ids")
            self._like(dlogprob, "dlogprob", torch.float32, ids.shape, dev)
        if dentropy is not None:
            if fwd.entropy is None:
                raise ValueError("dentropy needs a forward with entropy=True")
            self._like(dentropy, "dentropy", torch.float32, (M,), dev)
        self._like(fwd.lse, "the forward's lse", torch.float32, (M,), dev)
        self._check_dX(dX, X)

        def call(handle):
            out = torch.empty_like(X) if dX is None else dX
            saved = self._saved_of(fwd, M, n, handle)
            size = self._bwd_bytes(M, n, saved)
            ws = self._workspace(size, dev, handle)
            _check(_lib.lora_logprob_bwd(X.data_ptr(), M, byref(self.W.c_struct()), _ptr(ids), n, self.ignore_index,
                                         self.scale, fwd.lse.data_ptr(), _ptr(fwd.entropy), _ptr(dlogprob),
                                         _ptr(dentropy), _ptr(saved), out.data_ptr(), ws.data_ptr(), size,
                                         handle), "lora_logprob_bwd")
            self._used(fwd, saved)
            return out

        return self._run(call, X, stream, ids, dlogprob, dentropy, fwd.lse, fwd.entropy, fwd.saved, dX)


class LoraDistill(_HeadLayer):
    """Distillation from a teacher's top logits: per row, KL(q || softmax(X·Wᵀ/temperature))
    with q the softmax of the listed teacher logits over the same temperature, over a frozen bf16
    LM head ``W [V, D]``, without writing the ``[M, V]`` logits.

    ``forward(X, ids, teacher_logits)``: X bf16 [M, D]; ids int32 [M, n] and teacher_logits fp32
    [M, n] (n <= 128; log-probabilities serve as well, e.g. the ``top_ids`` and ``top_logprob`` of
    :class:`LoraTokenLogProbs` on the teacher's head with temperature 1: the temperature is applied
    here).  Entries whose id is ``ignore_index`` are left out; a row without any has loss 0 and no
    gradient.  ``save`` and ``slice_`` as for
    :class:`LoraTokenLogProbs`.  ``backward`` returns the gradient of Σ dloss·loss in X.
    """

    def _teacher(self, ids, teacher_logits, M, dev):
        n = self._ids(ids, M, dev, False)
        self._like(teacher_logits, "teacher_logits", torch.float32, (M, n), dev)
        return n

    def forward(self, X: torch.Tensor, ids: torch.Tensor, teacher_logits: torch.Tensor, save: bool = False,
                stream=None) -> DistillLoss:
        M, dev = self._hidden(X), X.device
        n = self._teacher(ids, teacher_logits, M, dev)

        def call(handle):
            loss = torch.empty(M, dtype=torch.float32, device=dev)
            out = DistillLoss(loss, torch.empty_like(loss), self._saved(M, n, dev) if save else None, n)
            size = self._bytes(_b.head_fwd_workspace_bytes, M, self.W.K, self.W.N, n, 0)
            ws = self._workspace(size, dev, handle)
            _check(_lib.lora_distill_fwd(X.data_ptr(), M, byref(self.W.c_struct()), ids.data_ptr(),
                                         teacher_logits.data_ptr(), n, self.ignore_index, self.scale,
                                         out.loss.data_ptr(), out.lse.data_ptr(), _ptr(out.saved), ws.data_ptr(),
                                         size, handle), "lora_distill_fwd")
            return self._mark(out, handle)

        return self._run(call, X, stream, ids, teacher_logits)

    def backward(self, X: torch.Tensor, ids: torch.Tensor, teacher_logits: torch.Tensor, fwd: DistillLoss,
                 dloss: torch.Tensor, dX=None, stream=None) -> torch.Tensor:
        M, dev = self._hidden(X), X.device
        n = self._teacher(ids, teacher_logits, M, dev)
        self._own(fwd, DistillLoss)
        self._like(dloss, "dloss", torch.float32, (M,), dev)
        self._like(fwd.lse, "the forward's lse", torch.float32, (M,), dev)
        self._check_dX(dX, X)

        def call(handle):
            out = torch.empty_like(X) if dX is None else dX
            saved = self._saved_of(fwd, M, n, handle)
            size = self._bwd_bytes(M, n, saved)
            ws = self._workspace(size, dev, handle)
            _check(_lib.lora_distill_bwd(X.data_ptr(), M, byref(self.W.c_struct()), ids.data_ptr(),
                                         teacher_logits.data_ptr(), n, self.ignore_index, self.scale,
                                         fwd.lse.data_ptr(), dloss.data_ptr(), _ptr(saved), out.data_ptr(),
                                         ws.data_ptr(), size, handle), "lora_distill_bwd")
            self._used(fwd, saved)
            return out

        return self._run(call, X, stream, ids, teacher_logits, dloss, fwd.lse, fwd.saved, dX)
