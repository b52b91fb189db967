"""The losses of a language model's head, over the C ABI of include/zero_loss.h:
what makes the gradients that the sharded step reduces.

A head is hidden states [tokens, dim] times a vocabulary matrix [vocab, dim].
Neither its logits nor their gradient is ever kept: both are made piece by piece
of the vocabulary inside the call.

  linear_xent(hidden, weight, target, ...)           -> loss [tokens], Saved
  linear_xent_grad(hidden, weight, target, saved, upstream, ...)
                                                     -> dhidden, dweight
  linear_distill(hidden, weight, index, logit, ...)  -> loss [tokens], Saved
  linear_distill_grad(hidden, weight, index, logit, saved, upstream, ...)
                                                     -> dhidden, dweight

linear_xent is softmax cross entropy against one target per token (with
ignore_index, label smoothing and z-loss); linear_distill the divergence of the
head's softmax from a teacher's top-K logits at a temperature. Losses are per
token and fp32; `upstream` is the gradient of the total with respect to each of
them, so the mean over n live tokens is upstream = 1 / n (a one-element tensor,
or an expanded one, broadcasts) and a loss scale multiplies it. A row with
nothing to learn from (ignore_index; no teacher entry) has loss 0 and no part in
any gradient, whatever it holds; a row whose target or teacher index is out of
range has loss NaN and no part in any gradient.

The gradients may be written to tensors the caller brings, among them views of a
worker's flat gradient buffer, where the sharded step reads them:

    head = zo.worker_grads(k)[i]                    # i: the head's place in parameters()
    loss, saved = linear_xent(h, weight, target)
    dh, _ = linear_xent_grad(h, weight, target, saved, 1.0 / n, dweight=head)
    h.backward(dh)                                  # the rest of the model

hidden, weight and their gradients are bf16, fp16 or fp32, all alike. Work is
enqueued on `stream` (torch's current one by default) and outputs are allocated
for it; inputs from another stream are the caller's to order, and to record. This
module checks and marshals arguments and allocates outputs and workspace from
torch; every step of the computation runs in libzero.so's HIP kernels.
"""
import ctypes as C
from dataclasses import dataclass

from . import _abi
from . import _raise, _stream_handle

__all__ = ["Saved", "linear_xent", "linear_xent_grad", "linear_distill", "linear_distill_grad",
           "loss_workspace_bytes"]

_DTYPES = {"torch.float32": _abi.ZERO_LOSS_F32, "torch.bfloat16": _abi.ZERO_LOSS_BF16,
           "torch.float16": _abi.ZERO_LOSS_F16}
_INDEX = {"torch.int32": _abi.ZERO_INDEX_I32, "torch.int64": _abi.ZERO_INDEX_I64}
_codes = {}  # the same by torch.dtype, filled as types are met: their names take long to form


def _code(dtype, table):
    at = (dtype, table is _INDEX)
    if at not in _codes:
        _codes[at] = table.get(str(dtype))
    return _codes[at]


@dataclass
class Saved:
    """What the loss leaves for its gradient: lse [tokens] and, for distillation,
    the student's logits at the teacher's entries [tokens, k]."""
    lse: object
    logit: object = None


def _matrix(x, what, dtype=None, shape=None):
    """A GPU matrix whose rows are contiguous, at any row stride."""
    import torch
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{what}: expected a torch.Tensor")
    if not x.is_cuda:
        raise ValueError(f"{what}: must be a GPU tensor")
    if x.dim() != 2:
        raise ValueError(f"{what}: expected two dimensions, got {tuple(x.shape)}")
    if shape is not None and tuple(x.shape) != tuple(shape):
        raise ValueError(f"{what}: shape {tuple(x.shape)}, expected {tuple(shape)}")
    if dtype is not None and x.dtype != dtype:
        raise ValueError(f"{what}: dtype {x.dtype}, expected {dtype}")
    if x.shape[1] > 1 and x.stride(1) != 1:
        raise ValueError(f"{what}: rows must be contiguous")
    return x


def _row_stride(x):
    """The stride between rows; a single row (or none) has whatever fits."""
    return max(x.stride(0), x.shape[1]) if x.shape[0] <= 1 else x.stride(0)


def _head(hidden, weight):
    _matrix(hidden, "hidden")
    _matrix(weight, "weight", hidden.dtype)
    if _code(hidden.dtype, _DTYPES) is None:
        raise ValueError(f"hidden: dtype {hidden.dtype}, expected bfloat16, float16 or float32")
    if hidden.shape[1] != weight.shape[1]:
        raise ValueError(f"hidden has {hidden.shape[1]} columns, weight {weight.shape[1]}")
    return _abi.zero_head(tokens=hidden.shape[0], vocab=weight.shape[0], dim=hidden.shape[1],
                          hidden=hidden.data_ptr() or None, hidden_stride=_row_stride(hidden),
                          weight=weight.data_ptr() or None, weight_stride=_row_stride(weight),
                          dtype=_code(hidden.dtype, _DTYPES), reserved=0)


def _index_dtype(x, what):
    code = _code(x.dtype, _INDEX)
    if code is None:
        raise ValueError(f"{what}: dtype {x.dtype}, expected int32 or int64")
    return code


def _xent_params(hidden, target, ignore_index, label_smoothing, z_loss):
    import torch
    if not isinstance(target, torch.Tensor):
        raise TypeError("target: expected a torch.Tensor")
    if not target.is_cuda:
        raise ValueError("target: must be a GPU tensor")
    if tuple(target.shape) != (hidden.shape[0],):
        raise ValueError(f"target: shape {tuple(target.shape)}, expected ({hidden.shape[0]},)")
    if not target.is_contiguous():
        raise ValueError("target: must be contiguous")
    return _abi.zero_xent_params(target=target.data_ptr() or None,
                                 index_dtype=_index_dtype(target, "target"), reserved=0,
                                 ignore_index=int(ignore_index),
                                 label_smoothing=float(label_smoothing), z_loss=float(z_loss))


def _distill_params(hidden, index, logit, temperature):
    _matrix(index, "index")
    _matrix(logit, "logit", shape=index.shape)
    if index.shape[0] != hidden.shape[0]:
        raise ValueError(f"index has {index.shape[0]} rows, hidden {hidden.shape[0]}")
    if _code(logit.dtype, _DTYPES) is None:
        raise ValueError(f"logit: dtype {logit.dtype}, expected bfloat16, float16 or float32")
    return _abi.zero_distill_params(index=index.data_ptr() or None, logit=logit.data_ptr() or None,
                                    index_stride=_row_stride(index),
                                    logit_stride=_row_stride(logit), k=index.shape[1],
                                    index_dtype=_index_dtype(index, "index"),
                                    logit_dtype=_code(logit.dtype, _DTYPES), reserved=0,
                                    temperature=float(temperature))


def _workspace_bytes(head, want_grad):
    out = C.c_size_t()
    st = _abi.load().zero_loss_workspace_bytes(C.byref(head), int(want_grad), C.byref(out))
    if st != _abi.ZERO_OK:
        _raise(st)
    return out.value


def loss_workspace_bytes(hidden, weight, want_grad: bool) -> int:
    """Device workspace bytes of one loss (or gradient) call on these tensors."""
    return _workspace_bytes(_head(hidden, weight), want_grad)


def _one_device(stream, *xs):
    """All tensors of a call (None left out) and a torch stream are on one GPU."""
    dev = xs[0].device
    for x in xs:
        if x is not None and x.device != dev:
            raise ValueError(f"all tensors of one call must be on one device, got {dev} and "
                             f"{x.device}")
    at = getattr(stream, "device", dev)
    if at != dev:
        raise ValueError(f"stream is on {at}, the tensors on {dev}")


class _NoContext:
    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


_NO_CONTEXT = _NoContext()


def _on_stream(stream, hidden):
    """A context on hidden's device in which torch allocates for `stream`: memory
    given back after the call is then reused in that stream's order."""
    import torch
    if stream is None:
        if torch.cuda.current_device() == hidden.device.index:
            return _NO_CONTEXT
        return torch.cuda.device(hidden.device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=hidden.device)
    return torch.cuda.stream(stream)  # also makes its device the current one


def _handle(stream, like):
    """The stream's hipStream_t. torch's current one is asked for directly where
    torch offers that: a Stream object takes 5 us to make."""
    if stream is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            return raw(like.device.index)
    return _stream_handle(stream, like)


def _check_workspace(workspace):
    import torch
    if workspace is not None and (not isinstance(workspace, torch.Tensor) or not workspace.is_cuda
                                  or not workspace.is_contiguous()):
        raise ValueError("workspace: must be a contiguous GPU tensor")


def _workspace(head, want_grad, workspace, like):
    import torch
    need = _workspace_bytes(head, want_grad)
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=like.device), need
    return workspace, workspace.numel() * workspace.element_size()


def linear_xent(hidden, weight, target, ignore_index: int = -100, label_smoothing: float = 0.0,
                z_loss: float = 0.0, workspace=None, stream=None):
    """Per-token cross entropy of softmax(hidden @ weight.T); returns (loss, Saved)."""
    import torch
    head = _head(hidden, weight)
    params = _xent_params(hidden, target, ignore_index, label_smoothing, z_loss)
    _check_workspace(workspace)
    _one_device(stream, hidden, weight, target, workspace)
    lib = _abi.load()
    with _on_stream(stream, hidden):
        loss = torch.empty(hidden.shape[0], dtype=torch.float32, device=hidden.device)
        lse = torch.empty_like(loss)
        ws, nbytes = _workspace(head, False, workspace, hidden)
        st = lib.zero_linear_xent(C.byref(head), C.byref(params), loss.data_ptr() or None,
                                  lse.data_ptr() or None, ws.data_ptr(), nbytes,
                                  _handle(stream, hidden))
    if st != _abi.ZERO_OK:
        _raise(st)
    return loss, Saved(lse)


def linear_distill(hidden, weight, index, logit, temperature: float = 1.0, workspace=None,
                   stream=None):
    """Per-token divergence of the head's softmax from the teacher's entries
    (index, logit) [tokens, k]; returns (loss, Saved)."""
    import torch
    head = _head(hidden, weight)
    params = _distill_params(hidden, index, logit, temperature)
    _check_workspace(workspace)
    _one_device(stream, hidden, weight, index, logit, workspace)
    lib = _abi.load()
    with _on_stream(stream, hidden):
        loss = torch.empty(hidden.shape[0], dtype=torch.float32, device=hidden.device)
        lse = torch.empty_like(loss)
        kept = torch.empty(index.shape, dtype=torch.float32, device=hidden.device)
        ws, nbytes = _workspace(head, False, workspace, hidden)
        st = lib.zero_linear_distill(C.byref(head), C.byref(params), loss.data_ptr() or None,
                                     lse.data_ptr() or None, kept.data_ptr() or None,
                                     ws.data_ptr(), nbytes, _handle(stream, hidden))
    if st != _abi.ZERO_OK:
        _raise(st)
    return loss, Saved(lse, kept)


def _check_saved(x, what, shape):
    import torch
    if not isinstance(x, torch.Tensor) or not x.is_cuda or not x.is_contiguous() \
            or x.dtype != torch.float32 or tuple(x.shape) != tuple(shape):
        raise ValueError(f"{what}: expected the contiguous fp32 GPU tensor {tuple(shape)} that the "
                         "loss returned")
    return x


def _upstream(upstream, hidden):
    """The fp32 upstream gradient and its stride; a number or one element broadcasts."""
    import torch
    tokens = hidden.shape[0]
    if not isinstance(upstream, torch.Tensor):
        upstream = torch.full((1,), float(upstream), dtype=torch.float32, device=hidden.device)
    if not upstream.is_cuda or upstream.dtype != torch.float32:
        raise ValueError("upstream: expected a float32 GPU tensor or a number")
    if upstream.numel() == 1 and upstream.dim() <= 1:
        return upstream, 0
    if tuple(upstream.shape) != (tokens,):
        raise ValueError(f"upstream: shape {tuple(upstream.shape)}, expected ({tokens},) or one "
                         "element")
    return upstream, upstream.stride(0)


def _grad(entry, hidden, weight, head, params, saved, extra, upstream, dhidden, dweight,
          need_dhidden, need_dweight, workspace, stream, tensors):
    import torch
    if not need_dhidden and not need_dweight:
        raise ValueError("nothing to do: need_dhidden and need_dweight are both False")
    if dhidden is not None:
        _matrix(dhidden, "dhidden", hidden.dtype, hidden.shape)
    if dweight is not None:
        _matrix(dweight, "dweight", weight.dtype, weight.shape)
    _check_saved(saved.lse, "saved.lse", (hidden.shape[0],))
    _check_workspace(workspace)
    _one_device(stream, hidden, weight, *tensors, saved.lse, dhidden, dweight, workspace,
                upstream if isinstance(upstream, torch.Tensor) else None)
    with _on_stream(stream, hidden):
        up, up_stride = _upstream(upstream, hidden)
        if need_dhidden and dhidden is None:
            dhidden = torch.empty(hidden.shape, dtype=hidden.dtype, device=hidden.device)
        if need_dweight and dweight is None:
            dweight = torch.empty(weight.shape, dtype=weight.dtype, device=weight.device)
        g = _abi.zero_head_grads(upstream=up.data_ptr() or None, upstream_stride=up_stride)
        if need_dhidden:
            g.dhidden, g.dhidden_stride = dhidden.data_ptr() or None, _row_stride(dhidden)
        if need_dweight:
            g.dweight, g.dweight_stride = dweight.data_ptr() or None, _row_stride(dweight)
        if hidden.shape[0] == 0 and not need_dweight:
            return dhidden, None  # no row: nothing is written
        ws, nbytes = _workspace(head, True, workspace, hidden)
        st = entry(C.byref(head), C.byref(params), saved.lse.data_ptr() or None, *extra,
                   C.byref(g), ws.data_ptr(), nbytes, _handle(stream, hidden))
    if st != _abi.ZERO_OK:
        _raise(st)
    return dhidden if need_dhidden else None, dweight if need_dweight else None


def linear_xent_grad(hidden, weight, target, saved: Saved, upstream, ignore_index: int = -100,
                     label_smoothing: float = 0.0, z_loss: float = 0.0, dhidden=None, dweight=None,
                     need_dhidden: bool = True, need_dweight: bool = True, workspace=None,
                     stream=None):
    """The gradients of sum_t upstream[t] * loss[t] with respect to hidden and
    weight, from the Saved of linear_xent with the same arguments; returns
    (dhidden, dweight), None for one that is not needed. Given dhidden or
    dweight tensors are written in place of new ones."""
    head = _head(hidden, weight)
    params = _xent_params(hidden, target, ignore_index, label_smoothing, z_loss)
    return _grad(_abi.load().zero_linear_xent_grad, hidden, weight, head, params, saved, (),
                 upstream, dhidden, dweight, need_dhidden, need_dweight, workspace, stream,
                 (target,))


def linear_distill_grad(hidden, weight, index, logit, saved: Saved, upstream,
                        temperature: float = 1.0, dhidden=None, dweight=None,
                        need_dhidden: bool = True, need_dweight: bool = True, workspace=None,
                        stream=None):
    """The gradients of sum_t upstream[t] * loss[t] with respect to hidden and
    weight, from the Saved of linear_distill with the same arguments; returns
    (dhidden, dweight) as linear_xent_grad does."""
    head = _head(hidden, weight)
    params = _distill_params(hidden, index, logit, temperature)
    _check_saved(saved.logit, "saved.logit", index.shape)
    return _grad(_abi.load().zero_linear_distill_grad, hidden, weight, head, params, saved,
                 (saved.logit.data_ptr() or None,), upstream, dhidden, dweight, need_dhidden,
                 need_dweight, workspace, stream, (index, logit, saved.logit))
