"""Torch conveniences of the 8-bit (E4M3, block-scaled) path.

``Fp8Weight``, ``Fp8Act`` and ``Fp8Workspace`` hold the buffers, ``fp8_linear``
and ``fp8_moe`` run the layers; all of them check shapes, types and devices and
then call the ``sharq_fp8_*`` functions.  Codes and scales are plain tensors:

    weight      codes float8_e4m3fn [D, K] or [E, D, K], scales float32
                [ceil(D/128), ceil(K/128)] (or with E in front)
    activation  codes float8_e4m3fn [T, K], scales float32 [T, ceil(K/128)]
                (stored column by column: stride(0) == 1)

Work runs on the device of the tensors and on `stream` (default: that device's
current stream); what a call allocates itself is allocated on that stream.
"""
import contextlib
import ctypes

import torch

import sparse_activation_quantization_b200 as _sq

__all__ = ["Fp8Weight", "Fp8Act", "Fp8Workspace", "fp8_linear", "fp8_moe"]

_F8 = torch.float8_e4m3fn


def _blocks(n):
    return -(-n // 128)


# The handle of a device's current stream and the current device, without building a Stream object (3 us of a call)
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _elsewhere(device, stream):
    """whether a call has to enter another device or stream first"""
    return stream is not None or _current_device() != device.index


@contextlib.contextmanager
def _on(device, stream):
    """Context in which a call's allocations and launches belong to `device` and `stream` (None: its current one)."""
    if stream is not None and stream.device != device:
        raise ValueError(f"stream of {stream.device}, tensors on {device}")
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                yield


def _call(name, device, stream, *args):
    """the sharq function `name` with these arguments and the stream's handle"""
    if _elsewhere(device, stream):
        with _on(device, stream):
            return _call(name, device, None, *args)
    status = getattr(_sq.lib(), name)(*args, _raw_stream(device.index))
    if status != 0:
        raise _sq.SharqError(status, name)


def _cuda(name, t, dtype, device=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != dtype:
        raise TypeError(f"{name} must be a {dtype} CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _rows(name, t, shape, dtype, device):
    """(pointer, row stride) of a 2-D tensor whose rows are contiguous"""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == device.index):
        _cuda(name, t, dtype, device)
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    ld, step = t.stride()
    if step != 1 and shape[1] > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return t.data_ptr(), ld if shape[0] > 1 else shape[1]


def _vector(name, t, n, dtype, device):
    if t is None:
        return None
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == device.index):
        _cuda(name, t, dtype, device)
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {n}")
    return t.data_ptr()


def _device(device):
    device = torch.device(device)
    if device.type != "cuda":
        raise ValueError(f"buffers lie on a CUDA device, got {device}")
    return torch.device("cuda", torch.cuda.current_device()) if device.index is None else device


class Fp8Weight:
    """E4M3 weight with one float32 scale per 128 x 128 block.

    Fp8Weight(W) quantizes a bf16 CUDA tensor [K, D] (or [E, K, D]) with
    sharq_fp8_pack_weight; Fp8Weight.from_parts(codes, scales) takes a
    checkpoint's tensors as they are."""

    def __init__(self, W, stream=None):
        _cuda("W", W, torch.bfloat16)
        if W.dim() not in (2, 3):
            raise ValueError("W must be [K, D] or [E, K, D]")
        E, K, D = (1, *W.shape) if W.dim() == 2 else W.shape
        lead = () if W.dim() == 2 else (E,)
        if _elsewhere(W.device, stream):
            with _on(W.device, stream):
                self._pack(W, lead, E, K, D)
        else:
            self._pack(W, lead, E, K, D)

    def _pack(self, W, lead, E, K, D):
        W = W.contiguous()
        self._set(W.new_empty((*lead, D, K), dtype=_F8),
                  W.new_empty((*lead, _blocks(D), _blocks(K)), dtype=torch.float32), E, K, D)
        _call("sharq_fp8_pack_weight", self.device, None, W.data_ptr(), self._ref)

    def _set(self, codes, scales, E, K, D):
        self.codes, self.scales = codes, scales
        self.E, self.K, self.D, self.device = E, K, D, codes.device
        self.view = _sq.SharqFp8Weight(codes.data_ptr(), scales.data_ptr(), K, D, E)
        self._ref = ctypes.byref(self.view)

    @classmethod
    def from_parts(cls, codes, scales):
        """codes float8_e4m3fn [D, K] or [E, D, K]; scales float32 [D/128, K/128]
        or [E, D/128, K/128] (rounded up).  Copied only if not contiguous."""
        _cuda("codes", codes, _F8)
        _cuda("scales", scales, torch.float32, codes.device)
        if codes.dim() not in (2, 3):
            raise ValueError("codes must be [D, K] or [E, D, K]")
        E, D, K = (1, *codes.shape) if codes.dim() == 2 else codes.shape
        if _sq.sharq_fp8_weight_bytes(K, D, E) == 0:
            raise _sq.SharqError(-2, "sharq_fp8_weight_bytes")
        if scales.shape != (*codes.shape[:-2], _blocks(D), _blocks(K)):
            raise ValueError(f"scales have shape {tuple(scales.shape)}")
        w = cls.__new__(cls)
        w._set(codes.contiguous(), scales.contiguous(), E, K, D)
        return w


class Fp8Act:
    """Prepared activation: codes [T, K] and scales [T, ceil(K/128)], the output
    of prep / prep_residual / prep_silu_mul and the input of fp8_linear."""

    def __init__(self, T, K, device="cuda"):
        n = _sq.sharq_fp8_act_bytes(T, K)
        if n == 0:
            raise _sq.SharqError(-2, "sharq_fp8_act_bytes")
        self.buf = torch.empty(n, dtype=torch.uint8, device=_device(device))
        view = _sq.sharq_fp8_act_view(self.buf.data_ptr(), T, K)
        kb, off = _blocks(K), view.scales - view.codes
        codes = self.buf[:T * K].view(_F8).view(T, K)
        scales = self.buf[off:off + 4 * kb * view.lds].view(torch.float32).view(kb, view.lds)[:, :T].t()
        self._set(codes, scales, view)

    def _set(self, codes, scales, view):
        self.codes, self.scales, self.view = codes, scales, view
        self.T, self.K, self.device = view.T, view.K, codes.device
        self._ref = ctypes.byref(view)

    @classmethod
    def from_parts(cls, codes, scales):
        """Codes float8_e4m3fn [T, K] and scales float32 [T, ceil(K/128)] from
        elsewhere.  Scales stored column by column (stride(0) == 1, stride(1) a
        multiple of 4 below 2^31, the last column as long as the others) are
        used as they are, others are copied."""
        _cuda("codes", codes, _F8)
        _cuda("scales", scales, torch.float32, codes.device)
        if codes.dim() != 2 or scales.shape != (codes.shape[0], _blocks(codes.shape[1])):
            raise ValueError(f"codes {tuple(codes.shape)} and scales {tuple(scales.shape)} do not belong together")
        T, K = codes.shape
        if _sq.sharq_fp8_act_bytes(T, K) == 0:
            raise _sq.SharqError(-2, "sharq_fp8_act_bytes")
        codes = codes.contiguous()
        lds = scales.stride(1)
        behind = scales.untyped_storage().nbytes() // 4 - scales.storage_offset()  # floats from the first scale on
        if (T > 1 and scales.stride(0) != 1) or lds < T or lds % 4 or lds >= 1 << 31 or scales.data_ptr() % 16 or \
                behind < _blocks(K) * lds:
            lds = -(-T // 4) * 4
            own = scales.new_empty(_blocks(K), lds)
            own[:, :T] = scales.t()
            scales = own[:, :T].t()
        a = cls.__new__(cls)
        a._set(codes, scales, _sq.SharqFp8Act(codes.data_ptr(), scales.data_ptr(), T, K, lds))
        return a

    def prep(self, X, gamma=None, eps=1e-5, stream=None):
        """Quantize X (bf16 [T, K]), normalised by its RMS when gamma is given."""
        x, ldx = _rows("X", X, (self.T, self.K), torch.bfloat16, self.device)
        g = _vector("gamma", gamma, self.K, torch.bfloat16, self.device)
        _call("sharq_fp8_prep", self.device, stream, x, ldx, g, eps, self._ref)
        return self

    def prep_residual(self, X, res, res_out=None, gamma=None, eps=1e-5, stream=None):
        """The same of h = bf16(X + res); h goes to res_out (which may be res
        itself) when given."""
        shape = (self.T, self.K)
        x, ldx = _rows("X", X, shape, torch.bfloat16, self.device)
        r, ldr = _rows("res", res, shape, torch.bfloat16, self.device)
        o, ldo = _rows("res_out", res_out, shape, torch.bfloat16, self.device) if res_out is not None else (None, 0)
        g = _vector("gamma", gamma, self.K, torch.bfloat16, self.device)
        _call("sharq_fp8_prep_residual", self.device, stream, x, ldx, r, ldr, o, ldo, g, eps, self._ref)
        return self

    def prep_silu_mul(self, gate, up, stream=None):
        """The same of silu(gate) * up; both may be views of one gate+up output."""
        shape = (self.T, self.K)
        g, ldg = _rows("gate", gate, shape, torch.bfloat16, self.device)
        u, ldu = _rows("up", up, shape, torch.bfloat16, self.device)
        _call("sharq_fp8_prep_silu_mul", self.device, stream, g, ldg, u, ldu, self._ref)
        return self


class Fp8Workspace:
    """Zeroed workspace of fp8_linear (its error word) or fp8_moe (error word and
    intermediate).  Calls that may run at the same time need one each."""

    def __init__(self, nbytes, device="cuda", stream=None):
        self.nbytes = int(nbytes)
        device = _device(device)
        with _on(device, stream):
            self.buf = torch.zeros(max(self.nbytes, 1), dtype=torch.uint8, device=device)
        self.ptr = self.buf.data_ptr()

    @classmethod
    def for_linear(cls, T, K, D, device="cuda", stream=None):
        n = _sq.sharq_fp8_linear_workspace_bytes(T, K, D)
        if n == 0:
            raise _sq.SharqError(-2, "sharq_fp8_linear_workspace_bytes")
        return cls(n, device, stream)

    @classmethod
    def for_moe(cls, T, topk, w13, w2, device="cuda", stream=None):
        n = _sq.sharq_fp8_moe_workspace_bytes(T, topk, w13.K, w2.K, w13.E)
        if n == 0:
            raise _sq.SharqError(-2, "sharq_fp8_moe_workspace_bytes")
        return cls(n, device, stream)

    def check(self, stream=None):
        """Synchronises and returns the error word of the calls that used it (0: none)."""
        with _on(self.buf.device, stream):
            return _sq.sharq_check_status(self.ptr, _raw_stream(self.buf.device.index))


def _workspace(ws, device):
    if ws.buf.device != device:
        raise ValueError(f"workspace on {ws.buf.device}, expected {device}")
    return ws


def fp8_linear(act, weight, out_dtype=None, out=None, ws=None, stream=None):
    """Y = X W through sharq_fp8_linear; act: Fp8Act, weight: Fp8Weight.  `out`
    (bf16 or float32, rows contiguous) may be a column slice of a wider tensor.
    ws: the Fp8Workspace whose check() tells of a wait that ran out; without one
    the call makes its own, whose error word is gone with it."""
    if weight.device != act.device:
        raise ValueError(f"weight on {weight.device}, activation on {act.device}")
    device = act.device
    if _elsewhere(device, stream):
        with _on(device, stream):
            return fp8_linear(act, weight, out_dtype, out, ws)
    out_dtype = out_dtype or (out.dtype if out is not None else torch.bfloat16)
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("the output is bf16 or float32")
    if out is None:
        out = act.codes.new_empty((act.T, weight.D), dtype=out_dtype)
        y, ldy = out.data_ptr(), weight.D
    else:
        y, ldy = _rows("out", out, (act.T, weight.D), out_dtype, device)
    ws = _workspace(ws, device) if ws is not None else Fp8Workspace.for_linear(act.T, act.K, weight.D, device)
    _call("sharq_fp8_linear", device, None, act._ref, weight._ref, y, ldy,
          _sq.SHARQ_OUT_F32 if out_dtype == torch.float32 else _sq.SHARQ_OUT_BF16, ws.ptr, ws.nbytes)
    return out


def fp8_moe(x, logits, w13, w2, topk, renormalize=True, out=None, ws=None, return_routing=False, stream=None):
    """A mixture-of-experts layer for a few tokens through sharq_fp8_moe.

    x: bf16 [T, H], T <= 64; logits: float32 [T, E], the router's output;
    w13: Fp8Weight of codes [E, 2 I, H], gate rows first; w2: of [E, H, I].
    Returns y (bf16 [T, H]; `out` may be x), with return_routing also the chosen
    experts (int32 [T, topk]) and their weights (float32 [T, topk]).  ws as in
    fp8_linear, from Fp8Workspace.for_moe."""
    device = w13.device
    if w2.device != device:
        raise ValueError(f"w2 on {w2.device}, w13 on {device}")
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be [T, H]")
    if _elsewhere(device, stream):
        with _on(device, stream):
            return fp8_moe(x, logits, w13, w2, topk, renormalize, out, ws, return_routing)
    T = x.shape[0]
    shape = (T, w13.K)
    xp, ldx = _rows("x", x, shape, torch.bfloat16, device)
    lp, ldl = _rows("logits", logits, (T, w13.E), torch.float32, device)
    if out is None:
        out = x.new_empty(shape)
        yp, ldy = out.data_ptr(), w13.K
    else:
        yp, ldy = _rows("out", out, shape, torch.bfloat16, device)
    ids = weights = ip = pp = None
    if return_routing:
        ids, weights = x.new_empty((T, topk), dtype=torch.int32), logits.new_empty((T, topk))
        ip, pp = ids.data_ptr(), weights.data_ptr()
    ws = _workspace(ws, device) if ws is not None else Fp8Workspace.for_moe(T, topk, w13, w2, device)
    _call("sharq_fp8_moe", device, None, xp, ldx, lp, ldl, T, topk, 1 if renormalize else 0, w13._ref, w2._ref, yp, ldy,
          ip, pp, ws.ptr, ws.nbytes)
    return (out, ids, weights) if return_routing else out
