"""Bindings of what stands around the linear attention in a layer: the elementwise gated recurrence (``dplr_gr_*``), and head
norms and rotary positions (``dplr_nr_*``). Argument marshalling only, as in ``dplr.py``."""

from __future__ import annotations

import ctypes
import math
import struct
from typing import Optional, Tuple

import torch

from .dplr import (DPLR_BF16, DPLR_ERR_INVALID_ARG, DPLR_F32, DPLR_OK, DplrError, RequestPlan, _int32, _need, _ref, _refuse,
                   _Slots, dplr_gr_desc, dplr_la_read_status, dplr_nr_desc, library)

GATES = {"log": 0, "sigmoid": 1}
INPUTS = {"plain": 0, "complement": 1, "unit": 2}
NORMS = {None: 0, "none": 0, "rms": 1, "l2": 2}
STATE_STEP = 64          # tokens between two states that a forward keeps (DPLR_GR_STATE_STEP)


def _type(dtype) -> int:
    if dtype in (torch.bfloat16, "bf16"):
        return DPLR_BF16
    if dtype in (torch.float32, "f32"):
        return DPLR_F32
    raise ValueError(f"unsupported dtype {dtype}")


def _torch_type(t: int) -> torch.dtype:
    return torch.bfloat16 if t == DPLR_BF16 else torch.float32


def _one_of(names: dict, value, what: str) -> int:
    if value not in names:
        raise ValueError(f"{what} is {value!r}, expected one of {[n for n in names if n is not None]}")
    return names[value]


# ----------------------------------------------------------------------------
# C-ABI mirrors (tensors as dplr_hd_tensor or None, everything else as pointers).
# ----------------------------------------------------------------------------

def make_gr_desc(in_dtype, B: int, T: int, D: int, gate="log", input="plain", gate_dtype=None) -> dplr_gr_desc:
    dt = _type(in_dtype)
    gt = dt if gate_dtype is None else _type(gate_dtype)
    return dplr_gr_desc(dt, gt, _one_of(GATES, gate, "gate"), _one_of(INPUTS, input, "input"), *_int32(B=B, T=T, D=D))


def dplr_gr_check(desc) -> int:
    return int(library().dplr_gr_check(ctypes.byref(desc)))


def dplr_gr_workspace_size(desc) -> int:
    return int(library().dplr_gr_workspace_size(ctypes.byref(desc)))


def dplr_gr_backward_workspace_size(desc) -> int:
    return int(library().dplr_gr_backward_workspace_size(ctypes.byref(desc)))


def dplr_gr_forward(desc, x, g, h0, y, h_T, states, workspace, ws_bytes, stream) -> int:
    return int(library().dplr_gr_forward(ctypes.byref(desc), _ref(x), _ref(g), h0, _ref(y), h_T, states, workspace, ws_bytes,
                                         stream))


def dplr_gr_backward(desc, x, g, h0, states, dy, dh_T, dx, dg, dh0, workspace, ws_bytes, stream) -> int:
    return int(library().dplr_gr_backward(ctypes.byref(desc), _ref(x), _ref(g), h0, states, _ref(dy), dh_T, _ref(dx),
                                          _ref(dg), dh0, workspace, ws_bytes, stream))


def dplr_gr_forward_packed(desc, R, n_slots, starts, token_slot, token_pos, x, g, h, y, workspace, ws_bytes, stream) -> int:
    return int(library().dplr_gr_forward_packed(ctypes.byref(desc), R, n_slots, starts, token_slot, token_pos, _ref(x),
                                                _ref(g), h, _ref(y), workspace, ws_bytes, stream))


def dplr_gr_decode_step(desc, n_slots, slots, x, g, h, y, status, stream) -> int:
    return int(library().dplr_gr_decode_step(ctypes.byref(desc), n_slots, slots, _ref(x), _ref(g), h, _ref(y), status,
                                             stream))


def make_nr_desc(in_dtype, B: int, T: int, q_heads: int, k_heads: int, d: int, rot: int, interleaved: bool = False,
                 norm=None, eps: float = 0.0, q_scale: float = 1.0, rot_scale: float = 1.0, grad_dtype=None) -> dplr_nr_desc:
    dt = _type(in_dtype)
    gt = dt if grad_dtype is None else _type(grad_dtype)
    sizes = _int32(B=B, T=T, q_heads=q_heads, k_heads=k_heads, d=d, rot=rot)
    return dplr_nr_desc(dt, gt, *sizes, int(bool(interleaved)), _one_of(NORMS, norm, "norm"), eps, q_scale, rot_scale)


def dplr_nr_check(desc) -> int:
    return int(library().dplr_nr_check(ctypes.byref(desc)))


def dplr_nr_turns(radians, n, turns) -> int:
    return int(library().dplr_nr_turns(radians, n, turns))


def dplr_nr_forward(desc, q, k, positions, pos_sb, pos_st, first_position, turns, q_weight, k_weight, q_out, k_out,
                    stream) -> int:
    return int(library().dplr_nr_forward(ctypes.byref(desc), _ref(q), _ref(k), positions, pos_sb, pos_st, first_position,
                                         turns, q_weight, k_weight, _ref(q_out), _ref(k_out), stream))


def dplr_nr_backward_workspace_size(desc) -> int:
    return int(library().dplr_nr_backward_workspace_size(ctypes.byref(desc)))


def dplr_nr_backward(desc, dq_out, dk_out, q, k, positions, pos_sb, pos_st, first_position, turns, q_weight, k_weight, dq,
                     dk, dq_weight, dk_weight, workspace, ws_bytes, stream) -> int:
    return int(library().dplr_nr_backward(ctypes.byref(desc), _ref(dq_out), _ref(dk_out), _ref(q), _ref(k), positions, pos_sb,
                                          pos_st, first_position, turns, q_weight, k_weight, _ref(dq), _ref(dk), dq_weight,
                                          dk_weight, workspace, ws_bytes, stream))


# ----------------------------------------------------------------------------
# Tensor-level wrappers.
# ----------------------------------------------------------------------------

class _Rows(_Slots):
    """_Slots whose last tensors, the outputs that the object owns, are filled in once."""

    def __init__(self, n: int, *outputs):
        super().__init__(n + len(outputs) // 4)
        self.refs = [ctypes.addressof(self.buf) + 32 * i for i in range(n + len(outputs) // 4)]
        self.fill(self.buf, 0, *(0,) * (4 * n), *outputs)
        self.fill = struct.Struct(f"={4 * n}q").pack_into


def _entry(name: str):
    """The C entry point `name` for prepared calls, which hand over addresses as plain numbers: ctypes takes 0.4 us less for
    ten of them than for pointers of their own types."""
    fn = library()[name]
    fn.argtypes = [t if t in (ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t) else ctypes.c_void_p
                   for t in getattr(library(), name).argtypes]
    fn.restype = ctypes.c_int
    return fn


class _Prepared:
    """What the prepared calls share: device, workspace, checks of tensors, the C call."""

    workspace: Optional[torch.Tensor] = None

    def _on(self, device):
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self._desc_ref = ctypes.addressof(self.desc)
        self._index = self.device.index

    def _work(self, nbytes: int, name: str):
        if nbytes == 0:
            raise DplrError(DPLR_ERR_INVALID_ARG, name)
        self.ws_bytes = nbytes
        self.workspace = torch.zeros(nbytes, dtype=torch.uint8, device=self.device)

    @staticmethod
    def _rows_of(shape, dtype):
        """What _at wants to know of a tensor: shape, type, elements in 16 bytes, and the strides that it has if contiguous
        (None where its rows would then not start on 16 bytes)."""
        unit, st = 16 // dtype.itemsize, [1]
        for n in reversed(shape[1:]):
            st.insert(0, n * st[0])
        return shape, dtype, unit, None if shape[-1] % unit else tuple(st)

    def _at(self, t, name, rows):
        """Address and strides of a tensor whose last axis is contiguous, in 16-byte steps."""
        shape, dtype, unit, dense = rows
        if t is None or t.dtype is not dtype or t.shape != shape or t.get_device() != self._index:
            _refuse(t, name, self.device, dtype, shape)
        p = t.data_ptr()
        if dense is not None and not p & 15 and t.is_contiguous():
            return p, dense
        st = t.stride()
        if t.numel():
            if p & 15 or (st[-1] != 1 and shape[-1] > 1):
                _refuse(t, name, self.device, dtype, shape)
            for n, s in zip(shape[:-1], st):
                if n > 1 and (s <= 0 or s % unit):
                    _refuse(t, name, self.device, dtype, shape)
        return p, st

    def _plain(self, t, name, shape, dtype=torch.float32):
        """Address of a contiguous tensor, or None."""
        if t is None:
            return None
        if t.dtype is not dtype or t.shape != shape or t.get_device() != self._index or not t.is_contiguous():
            _need(t, name, self.device, dtype, shape)
        return t.data_ptr()

    def _call(self, fn, name, stream, *args):
        i = self._index
        s = stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(i)
        if torch._C._cuda_getDevice() == i:
            st = fn(self._desc_ref, *args, s)
        else:
            with torch.cuda.device(i):
                st = fn(self._desc_ref, *args, s)
        if st != DPLR_OK:
            raise DplrError(st, name)

    def device_status(self, clear: bool = False) -> int:
        """The workspace's device status word (0, DPLR_ERR_TIMEOUT after a bounded wait gave up, or DPLR_ERR_INVALID_ARG
        after a ragged forward found a slot out of range), read synchronously through dplr_la_read_status."""
        with torch.cuda.device(self.device):
            s = torch.cuda.current_stream(self.device)
            st, word = dplr_la_read_status(self.workspace.data_ptr(), self.ws_bytes, clear, s.cuda_stream)
        if st != DPLR_OK:
            raise DplrError(st, "dplr_la_read_status")
        return word


class _Recurrence(_Prepared):
    def _setup(self, in_dtype, B, T, D, gate, input, gate_dtype, device):
        self.desc = make_gr_desc(in_dtype, B, T, D, gate, input, gate_dtype)
        st = dplr_gr_check(self.desc)
        if st != DPLR_OK:
            raise DplrError(st, "dplr_gr_check")
        self.B, self.T, self.D = self.desc.B, self.desc.T, self.desc.D
        self._one = (self.B, self.D)
        self.in_dtype, self.gate_dtype = _torch_type(self.desc.in_dtype), _torch_type(self.desc.gate_dtype)
        self._inputs(self.B, self.T, self.D)
        self._on(device)

    def _inputs(self, *shape):
        self._x, self._g = self._rows_of(shape, self.in_dtype), self._rows_of(shape, self.gate_dtype)

    def _rows(self, lead, dtype):
        """Zeros [*lead, D] whose rows start on 16 bytes."""
        unit = 16 // dtype.itemsize
        return torch.zeros((*lead, self.D + -self.D % unit), dtype=dtype, device=self.device)[..., :self.D]


class GatedRecurrence(_Recurrence):
    """Prepared forward of the elementwise gated recurrence (dplr_gr_forward): h_t = a_t h_{t-1} + b_t, y_t = h_t, with
    a = exp(g) (gate="log", g <= 0) or sigmoid(g) ("sigmoid") and b = x (input="plain"), (1 - a) x ("complement") or
    sqrt(1 - a^2) x ("unit"). Owns y [B,T,D] (the inputs' type; rows padded to 16 bytes where D does not fill them), h_T
    [B,D] fp32, with `keep_states` the states that a backward starts from, and the workspace, so that repeated calls
    allocate nothing. `gate_dtype`: the inputs' type or torch.float32."""

    def __init__(self, in_dtype, B: int, T: int, D: int, gate: str = "log", input: str = "plain", gate_dtype=None,
                 keep_states: bool = False, device: Optional[torch.device] = None):
        self._setup(in_dtype, B, T, D, gate, input, gate_dtype, device)
        with torch.cuda.device(self.device):
            self._work(dplr_gr_workspace_size(self.desc), "dplr_gr_workspace_size")
            self.y = self._rows((B, T), self.in_dtype)
            self.h_T = torch.zeros((B, D), dtype=torch.float32, device=self.device)
            self.states = torch.zeros((B, -(-T // STATE_STEP), D), dtype=torch.float32,
                                      device=self.device) if keep_states else None
        st = self.y.stride()
        self._fn, self._slots = _entry("dplr_gr_forward"), _Rows(2, self.y.data_ptr(), st[0], 0, st[1])
        self._own = (self.h_T.data_ptr(), None if self.states is None else self.states.data_ptr(), self.workspace.data_ptr(),
                     self.ws_bytes)

    def __call__(self, x, gate, h0=None, stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """x, gate [B,T,D] strided as they are (the channels contiguous, rows on 16 bytes); h0 [B,D] fp32, which may be
        this object's h_T. Returns y and h_T."""
        px, sx = self._at(x, "x", self._x)
        pg, sg = self._at(gate, "gate", self._g)
        ph = self._plain(h0, "h0", self._one)
        f = self._slots
        with f.turn:
            f(px, sx[0], 0, sx[1], pg, sg[0], 0, sg[1])
            r = f.refs
            self._call(self._fn, "dplr_gr_forward", stream, r[0], r[1], ph, r[2], *self._own)
        return self.y, self.h_T


class GatedRecurrenceBackward(_Recurrence):
    """Prepared backward of GatedRecurrence (dplr_gr_backward): owns the workspace and the gradients, x in the inputs' type,
    gate in the gates' and h0 in fp32."""

    def __init__(self, in_dtype, B: int, T: int, D: int, gate: str = "log", input: str = "plain", gate_dtype=None,
                 device: Optional[torch.device] = None):
        self._setup(in_dtype, B, T, D, gate, input, gate_dtype, device)
        with torch.cuda.device(self.device):
            self._work(dplr_gr_backward_workspace_size(self.desc), "dplr_gr_backward_workspace_size")
            self.grads = {"x": self._rows((B, T), self.in_dtype), "gate": self._rows((B, T), self.gate_dtype),
                          "h0": torch.zeros((B, D), dtype=torch.float32, device=self.device)}
        G = self.grads
        own = [v for n in ("x", "gate") for v in (G[n].data_ptr(), G[n].stride(0), 0, G[n].stride(1))]
        self._fn, self._slots = _entry("dplr_gr_backward"), _Rows(3, *own)
        self._own = (G["h0"].data_ptr(), self.workspace.data_ptr(), self.ws_bytes)

    def __call__(self, dy, dh_T, x, gate, h0=None, states=None, stream: Optional[torch.cuda.Stream] = None) -> dict:
        """Gradients of GatedRecurrence's inputs (a dict, also kept in .grads) given dy [B,T,D] in the inputs' type and dh_T
        [B,D] (fp32 or None: zero). `states`: those that the forward of the same x, gate and h0 kept; without them they are
        formed again, which reads x and gate once more."""
        one = self._one
        at = [self._at(x, "x", self._x), self._at(gate, "gate", self._g), self._at(dy, "dy", self._x)]
        p0, ps = self._plain(h0, "h0", one), self._plain(states, "states", (self.B, -(-self.T // STATE_STEP), self.D))
        pT, f = self._plain(dh_T, "dh_T", one), self._slots
        with f.turn:
            f(*[v for p, st in at for v in (p, st[0], 0, st[1])])
            r = f.refs
            self._call(self._fn, "dplr_gr_backward", stream, r[0], r[1], p0, ps, r[2], pT, r[3], r[4], *self._own)
        return self.grads


class GatedRecurrencePacked(_Recurrence):
    """Prepared forward of a ragged batch (dplr_gr_forward_packed) on a pool of states: `plan` (a RequestPlan; one is made if
    none is given) says which rows belong to which request, and may be the one that a HeadDecayPacked uses. Owns the output y
    [capacity,D] (rows behind the last token stay as they were) and the workspace."""

    def __init__(self, in_dtype, requests: int, capacity: int, slots: int, D: int, gate: str = "log", input: str = "plain",
                 gate_dtype=None, plan: Optional[RequestPlan] = None, device: Optional[torch.device] = None):
        self._setup(in_dtype, 1, capacity, D, gate, input, gate_dtype, device)
        self._inputs(self.T, self.D)
        if plan is None:
            plan = RequestPlan(requests, capacity, slots, device=self.device)
        elif (plan.R, plan.capacity, plan.n_slots, plan.device) != (requests, capacity, slots, self.device):
            raise ValueError("the plan is for another number of requests, capacity, slots or device")
        self.plan, self.n_slots = plan, plan.n_slots
        with torch.cuda.device(self.device):
            self._work(dplr_gr_workspace_size(self.desc), "dplr_gr_workspace_size")
            self.y = self._rows((capacity,), self.in_dtype)
        self._fn, self._slots = _entry("dplr_gr_forward_packed"), _Rows(2, self.y.data_ptr(), 0, 0, self.y.stride(0))
        self._own = (self.workspace.data_ptr(), self.ws_bytes)
        self._tables = (plan.starts.data_ptr(), plan.token_slot.data_ptr(), plan.token_pos.data_ptr())

    def __call__(self, x, gate, S, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """x, gate [capacity,D]; S [slots,D] fp32 is updated in place."""
        p = self.plan
        if not hasattr(p, "slots"):
            raise ValueError("call the plan first: it makes the tables")
        if S is None:
            raise ValueError("S is required")
        px, sx = self._at(x, "x", self._x)
        pg, sg = self._at(gate, "gate", self._g)
        pS = self._plain(S, "S", (self.n_slots, self.D))
        f = self._slots
        with f.turn:
            f(px, 0, 0, sx[0], pg, 0, 0, sg[0])
            r = f.refs
            self._call(self._fn, "dplr_gr_forward_packed", stream, p.R, self.n_slots, *self._tables, r[0], r[1], pS, r[2],
                       *self._own)
        return self.y


class GatedRecurrenceDecode(_Recurrence):
    """Prepared one-token step for `rows` rows on a pool of states (dplr_gr_decode_step): owns the output y [rows,D]."""

    def __init__(self, in_dtype, rows: int, D: int, slots: int, gate: str = "log", input: str = "plain", gate_dtype=None,
                 device: Optional[torch.device] = None):
        self._setup(in_dtype, rows, 1, D, gate, input, gate_dtype, device)
        self.n_slots, = _int32(slots=int(slots))
        self.y = self._rows((rows,), self.in_dtype)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._fn, self._slots = _entry("dplr_gr_decode_step"), _Rows(2, self.y.data_ptr(), self.y.stride(0), 0, 0)
        self._inputs(self.B, self.D)
        self._pool, self._one = (self.n_slots, self.D), (self.B,)
        self._status = self.status.data_ptr()

    def device_status(self, clear: bool = False) -> int:
        """DPLR_ERR_INVALID_ARG if a row's slot was out of range or an earlier row's since the word was cleared."""
        word = int(self.status.item())
        if clear:
            self.status.zero_()
        return word

    def __call__(self, x, gate, S, slots, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """x, gate [rows,D]; S [slots,D] fp32 is updated in place; slots [rows] int32: each row's state, -1 for a row
        without one."""
        if S is None:
            raise ValueError("S is required")
        if slots is None:
            raise ValueError("slots is required")
        px, sx = self._at(x, "x", self._x)
        pg, sg = self._at(gate, "gate", self._g)
        pS, pi = self._plain(S, "S", self._pool), self._plain(slots, "slots", self._one, torch.int32)
        f = self._slots
        with f.turn:
            f(px, sx[0], 0, 0, pg, sg[0], 0, 0)
            r = f.refs
            self._call(self._fn, "dplr_gr_decode_step", stream, self.n_slots, pi, r[0], r[1], pS, r[2], self._status)
        return self.y


def rotary_frequencies(rot: int, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                       trained: Optional[int] = None, slow: float = 1.0, fast: float = 32.0) -> torch.Tensor:
    """Frequencies (radians a position, float64 [rot / 2]) base^(-2i / rot), scaled to reach `factor` times as far:
    "linear" divides all by the factor; "base" stretches the base so that the slowest is divided by it and the fastest kept;
    "parts" divides those that make fewer than `slow` turns over the `trained` length, keeps those that make more than
    `fast`, and goes from one to the other in proportion to the turns between."""
    if rot < 0 or rot % 2:
        raise ValueError(f"rot is {rot}, expected an even number")
    if not base > 0 or not factor > 0:
        raise ValueError("base and factor must be positive")
    if scaling == "base" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    elif scaling == "parts":
        if trained is None or not trained > 0 or not fast > slow:
            raise ValueError("scaling by parts needs the trained length and slow < fast")
        keep = [min(max((trained * x / (2 * math.pi) - slow) / (fast - slow), 0.0), 1.0) for x in f]
        f = [x * (k + (1 - k) / factor) for x, k in zip(f, keep)]
    elif scaling not in (None, "none", "base"):
        raise ValueError(f"scaling is {scaling!r}, expected 'linear', 'base' or 'parts'")
    return torch.tensor(f, dtype=torch.float64)


class _Rotary(_Prepared):
    def _setup(self, in_dtype, B, T, q_heads, k_heads, d, frequencies, interleaved, norm, eps, q_scale, rot_scale,
               token_major, grad_dtype, device):
        f = torch.as_tensor(frequencies, dtype=torch.float64).detach().cpu().contiguous()
        if f.dim() != 1:
            raise ValueError("frequencies must be one-dimensional")
        self.desc = make_nr_desc(in_dtype, B, T, q_heads, k_heads, d, 2 * f.numel(), interleaved, norm, eps, q_scale,
                                 rot_scale, grad_dtype)
        st = dplr_nr_check(self.desc)
        if st != DPLR_OK:
            raise DplrError(st, "dplr_nr_check")
        self.B, self.T, self.Hq, self.Hk, self.d = (getattr(self.desc, n) for n in ("B", "T", "Hq", "Hk", "d"))
        self.in_dtype, self.grad_dtype = _torch_type(self.desc.in_dtype), _torch_type(self.desc.grad_dtype)
        self._on(device)
        turns = torch.zeros(max(f.numel(), 1), dtype=torch.int64)
        st = dplr_nr_turns(f.data_ptr() if f.numel() else None, f.numel(), turns.data_ptr())
        if st != DPLR_OK:
            raise DplrError(st, "dplr_nr_turns")
        self.turns = turns.to(self.device)
        self._turns = self.turns.data_ptr()
        self._in, self._dout = ([self._rows_of((self.B, h, self.T, self.d), t) for h in (self.Hq, self.Hk)]
                                for t in (self.in_dtype, self.grad_dtype))
        self._pos_shape, self._w_shape = (self.B, self.T), (self.d,)
        make = self._token_major if token_major else self._head_major
        self._out = [make(self.Hq), make(self.Hk) if self.Hk else None]

    def _head_major(self, heads):
        return torch.zeros((self.B, heads, self.T, self.d), dtype=self.in_dtype, device=self.device)

    def _token_major(self, heads):
        return torch.zeros((self.B, self.T, heads, self.d), dtype=self.in_dtype, device=self.device).transpose(1, 2)

    def _pair(self, q, k, names, rows):
        """Addresses and strides of a tensor of queries and one of keys."""
        p, s = self._at(q, names[0], rows[0])
        if not self.Hk:
            if k is not None:
                raise ValueError(f"{names[1]} is given, but there are no key heads")
            return (p, s[0], s[1], s[2], 0, 0, 0, 0)
        pk, sk = self._at(k, names[1], rows[1])
        return (p, s[0], s[1], s[2], pk, sk[0], sk[1], sk[2])

    def _outputs(self):
        q, k = self._out
        s = q.stride()
        if k is None:
            return (q.data_ptr(), s[0], s[1], s[2], 0, 0, 0, 0)
        sk = k.stride()
        return (q.data_ptr(), s[0], s[1], s[2], k.data_ptr(), sk[0], sk[1], sk[2])

    def _positions(self, t, first):
        if t is None:
            first, = _int32(first_position=first)
            return None, 0, 0, first
        if t.dtype is not torch.int32 or t.shape != self._pos_shape or t.get_device() != self._index:
            _refuse(t, "positions", self.device, torch.int32, self._pos_shape)
        sb, st = t.stride()
        return t.data_ptr(), sb, st, 0


class Rotary(_Rotary):
    """Prepared rotary positions for queries and keys (dplr_nr_forward without a norm): owns the outputs q [B,Hq,T,d] and k
    [B,Hk,T,d] (the inputs' type; stored with the tokens before the heads if `token_major`; k None without key heads).
    `frequencies`: radians a position for each pair, float64 (rotary_frequencies); 2 len(frequencies) features of each head
    are rotated. Pairs are halves apart, or neighbours if `interleaved`. Rotated features are multiplied by `rot_scale`, all
    features of queries by `q_scale`."""

    def __init__(self, in_dtype, B: int, T: int, q_heads: int, k_heads: int, d: int, frequencies, interleaved: bool = False,
                 q_scale: float = 1.0, rot_scale: float = 1.0, token_major: bool = False,
                 device: Optional[torch.device] = None):
        self._prepare(in_dtype, B, T, q_heads, k_heads, d, frequencies, interleaved, None, 0.0, q_scale, rot_scale,
                      token_major, device)

    def _prepare(self, in_dtype, B, T, q_heads, k_heads, d, frequencies, interleaved, norm, eps, q_scale, rot_scale,
                 token_major, device):
        self._setup(in_dtype, B, T, q_heads, k_heads, d, frequencies, interleaved, norm, eps, q_scale, rot_scale,
                    token_major, None, device)
        self.q, self.k = self._out
        self._fn, self._slots = _entry("dplr_nr_forward"), _Rows(2, *self._outputs())

    def __call__(self, q, k, positions=None, first_position: int = 0,
                 stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
        """q [B,Hq,T,d], k [B,Hk,T,d] strided as they are; positions int32 [B,T] (any strides; a negative one is a row
        without a token, whose outputs stay as they were), or None: first_position + t."""
        return self._run(q, k, positions, first_position, None, None, stream)

    def _run(self, q, k, positions, first, wq, wk, stream):
        rows = self._pair(q, k, ("q", "k"), self._in)
        at = self._positions(positions, first)
        f = self._slots
        with f.turn:
            f(*rows)
            r = f.refs
            self._call(self._fn, "dplr_nr_forward", stream, r[0], r[1], *at, self._turns, wq, wk, r[2], r[3])
        return self.q, self.k


class NormRotary(Rotary):
    """Prepared norms of queries and keys with the rotation in the same pass (dplr_nr_forward): each head is divided by its
    root mean square (norm="rms") or its length ("l2"), eps inside the root, times a weight a feature if `weights`, then
    rotated as by Rotary."""

    def __init__(self, in_dtype, B: int, T: int, q_heads: int, k_heads: int, d: int, frequencies, norm: str = "rms",
                 eps: float = 1e-6, weights: bool = True, interleaved: bool = False, q_scale: float = 1.0,
                 rot_scale: float = 1.0, token_major: bool = False, device: Optional[torch.device] = None):
        if norm not in ("rms", "l2"):
            raise ValueError(f"norm is {norm!r}, expected 'rms' or 'l2'")
        self._prepare(in_dtype, B, T, q_heads, k_heads, d, frequencies, interleaved, norm, eps, q_scale, rot_scale,
                      token_major, device)
        self.weights = bool(weights)

    def __call__(self, q, k, positions=None, first_position: int = 0, q_weight=None, k_weight=None,
                 stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
        """As Rotary; q_weight and k_weight fp32 [d] with `weights`."""
        return self._run(q, k, positions, first_position, *_weights(self, q_weight, k_weight), stream)


def _weights(self, q_weight, k_weight):
    """Addresses of the weights that a call needs."""
    out = []
    for t, name, heads in ((q_weight, "q_weight", self.Hq), (k_weight, "k_weight", self.Hk)):
        if (t is None) == (self.weights and heads > 0):
            raise ValueError(f"{name} is required" if t is None else f"{name} is given to a call without such weights")
        out.append(self._plain(t, name, self._w_shape))
    return out


class RotaryBackward(_Rotary):
    """Prepared backward of Rotary (dplr_nr_backward without a norm): owns the gradients q and k (a dict). `grad_dtype`: the
    type of the gradients that come in, the inputs' or torch.float32."""

    def __init__(self, in_dtype, B: int, T: int, q_heads: int, k_heads: int, d: int, frequencies, interleaved: bool = False,
                 q_scale: float = 1.0, rot_scale: float = 1.0, token_major: bool = False, grad_dtype=None,
                 device: Optional[torch.device] = None):
        self._prepare(in_dtype, B, T, q_heads, k_heads, d, frequencies, interleaved, None, 0.0, q_scale, rot_scale,
                      token_major, grad_dtype, device)

    def _prepare(self, in_dtype, B, T, q_heads, k_heads, d, frequencies, interleaved, norm, eps, q_scale, rot_scale,
                 token_major, grad_dtype, device):
        self._setup(in_dtype, B, T, q_heads, k_heads, d, frequencies, interleaved, norm, eps, q_scale, rot_scale,
                    token_major, grad_dtype, device)
        with torch.cuda.device(self.device):
            self._work(dplr_nr_backward_workspace_size(self.desc), "dplr_nr_backward_workspace_size")
        self.grads = {"q": self._out[0], "k": self._out[1]}
        self._fn, self._slots = _entry("dplr_nr_backward"), _Rows(4, *self._outputs())
        self._own = (self.workspace.data_ptr(), self.ws_bytes)

    def __call__(self, dq, dk, positions=None, first_position: int = 0,
                 stream: Optional[torch.cuda.Stream] = None) -> dict:
        """Gradients of Rotary's inputs given those of its outputs, dq [B,Hq,T,d] and dk [B,Hk,T,d]; zero in rows without a
        token."""
        return self._run(dq, dk, None, positions, first_position, None, None, None, None, stream)

    def _run(self, dq, dk, inputs, positions, first, wq, wk, dwq, dwk, stream):
        rows = self._pair(dq, dk, ("dq", "dk"), self._dout)
        rows += (0,) * 8 if inputs is None else self._pair(*inputs, ("q", "k"), self._in)
        at = self._positions(positions, first)
        f = self._slots
        with f.turn:
            f(*rows)
            r = f.refs
            self._call(self._fn, "dplr_nr_backward", stream, r[0], r[1], r[2], r[3], *at, self._turns, wq, wk, r[4], r[5], dwq,
                       dwk, *self._own)
        return self.grads


class NormRotaryBackward(RotaryBackward):
    """Prepared backward of NormRotary (dplr_nr_backward): owns the gradients q and k, and with `weights` q_weight and
    k_weight (fp32 [d], summed over batch, heads and tokens in a fixed order)."""

    def __init__(self, in_dtype, B: int, T: int, q_heads: int, k_heads: int, d: int, frequencies, norm: str = "rms",
                 eps: float = 1e-6, weights: bool = True, interleaved: bool = False, q_scale: float = 1.0,
                 rot_scale: float = 1.0, token_major: bool = False, grad_dtype=None,
                 device: Optional[torch.device] = None):
        if norm not in ("rms", "l2"):
            raise ValueError(f"norm is {norm!r}, expected 'rms' or 'l2'")
        self._prepare(in_dtype, B, T, q_heads, k_heads, d, frequencies, interleaved, norm, eps, q_scale, rot_scale,
                      token_major, grad_dtype, device)
        self.weights = bool(weights)
        if self.weights:
            for n, heads in (("q_weight", self.Hq), ("k_weight", self.Hk)):
                self.grads[n] = torch.zeros(self.d, dtype=torch.float32, device=self.device) if heads else None

    def __call__(self, dq, dk, q, k, positions=None, first_position: int = 0, q_weight=None, k_weight=None,
                 stream: Optional[torch.cuda.Stream] = None) -> dict:
        """Gradients of NormRotary's inputs given those of its outputs, and its inputs; zero in rows without a token, which add
        nothing to those of the weights."""
        wq, wk = _weights(self, q_weight, k_weight)
        dw = [None if self.grads.get(n) is None else self.grads[n].data_ptr() for n in ("q_weight", "k_weight")]
        return self._run(dq, dk, (q, k), positions, first_position, wq, wk, *dw, stream)
