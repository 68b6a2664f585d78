"""AdamW over a list of tensors that stay where they are, with 32-bit or 8-bit
states: the library's ``zero_multi_*`` calls with the buffers they need.

:class:`MultiAdamW` is for parameters outside a :class:`.engine.ZeroStep`'s
flat buffer (replicated norms and biases, a model trained without ZeRO) and
for groups of tensors with learning rates and weight decays of their own.  One
step is one launch, or two where a clip threshold or a loss scaler makes the
update wait for the global norm.  :class:`StateCodec8` turns 32-bit states
into the 8-bit form and back.

8-bit states hold m as E4M3 and v as E5M2 numbers, one power of two (E8M0) per
32 consecutive elements of a tensor: ``code.float() * scale.float()`` is the
value.  The calls are asynchronous on the object's stream (torch's current one
by default), as everywhere in this package.
"""
from __future__ import annotations

import ctypes
from contextlib import nullcontext
from typing import List, Optional, Sequence

import torch

from . import binding as B
from .engine import AdamW, read_step_state

BLOCK = 32
_GRAD = {torch.bfloat16: B.ZERO_BF16, torch.float16: B.ZERO_FP16, torch.float32: B.ZERO_FP32}
_PARAM = {torch.bfloat16: B.ZERO_BF16, torch.float16: B.ZERO_FP16}
M8, V8, SCALE8 = torch.float8_e4m3fn, torch.float8_e5m2, torch.float8_e8m0fnu


def _check_list(name: str, xs: Sequence[torch.Tensor], numels: Sequence[int], dtypes, device) -> None:
    if len(xs) != len(numels):
        raise ValueError("%s: expected %d tensors, got %d" % (name, len(numels), len(xs)))
    index, dtype = device.index, xs[0].dtype
    if device.type == "cuda" and dtype in dtypes and all(x.numel() == n and x.dtype is dtype and x.get_device() == index and
                                                         x.is_contiguous() for x, n in zip(xs, numels)):
        return
    for i, (x, n) in enumerate(zip(xs, numels)):     # what it is
        if x.numel() != n:
            raise ValueError("%s[%d]: expected %d elements, got %d" % (name, i, n, x.numel()))
        if x.dtype not in dtypes or x.dtype != dtype:
            raise ValueError("%s[%d]: dtype %s (need %s, one for the list)" % (name, i, x.dtype, "/".join(map(str, dtypes))))
        if not x.is_contiguous():
            raise ValueError("%s[%d] is not contiguous" % (name, i))
    raise ValueError("%s: the list's tensors are on CUDA device %s" % (name, index))


def scale_count(numel: int) -> int:
    """Scale bytes of one 8-bit state of a tensor."""
    return -(-numel // BLOCK)


def _slices(numels: Sequence[int], dtype, device) -> List[torch.Tensor]:
    """Zeroed tensors of these sizes in one allocation, each on a 256-byte boundary."""
    size = torch.empty(0, dtype=dtype).element_size()
    step = 256 // size
    starts, at = [], 0
    for n in numels:
        starts.append(at)
        at += -(-n // step) * step
    flat = torch.zeros(at * size, dtype=torch.uint8, device=device).view(dtype)
    return [flat[a:a + n] for a, n in zip(starts, numels)]


def used_on(stream: Optional[torch.cuda.Stream], *lists) -> None:
    """Tell torch's allocator that kernels on an object's own stream use these
    tensors: memory whose last reference goes while they run is given out again
    only after them."""
    if stream is not None:
        for xs in lists:
            for x in xs or ():
                x.record_stream(stream)


class BoundList:
    """A bound ``zero_multi`` and its workspace."""

    def __init__(self, numels, group_of_tensor, n_groups, grad_dtype, param_dtype, device):
        self.M = B.zero_multi_init(numels, group_of_tensor, n_groups, grad_dtype, param_dtype)
        self.info = B.zero_multi_query(self.M)
        self.workspace = torch.zeros(self.info.workspace_bytes, dtype=torch.uint8, device=device)

    def error_word(self) -> torch.Tensor:
        """Where the codec's kernels report errors: the fourth word of the
        workspace, what zero_multi_device_error reads."""
        return self.workspace[12:16].view(torch.int32)

    def bind(self, stream, **arrays):
        # the workspace's zero fill, and whatever made the tensors, ran on the current stream
        stream.wait_stream(torch.cuda.current_stream(self.workspace.device))
        B.zero_multi_bind(self.M, self.workspace, stream, **arrays)


_current_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _device(index: int):
    """The library launches on the current device: with this one current."""
    return nullcontext() if _current_device() == index else torch.cuda.device(index)


class StateCodec8:
    """The 32-bit states ``m``, ``v`` (lists of fp32 tensors) and the 8-bit
    ones ``m8`` (float8_e4m3fn), ``v8`` (float8_e5m2), ``m8_scale`` and
    ``v8_scale`` (float8_e8m0fnu, one per 32 elements) of the same tensors:
    :meth:`encode` writes the second from the first, :meth:`decode` the first
    from the second.  A kernel whose waits ran out leaves elements unwritten
    and an error: :meth:`check` raises then, :meth:`report` hands it on."""

    def __init__(self, m, v, m8, m8_scale, v8, v8_scale, stream: Optional[torch.cuda.Stream] = None):
        if not len(m):
            raise ValueError("no tensors")
        numels = [x.numel() for x in m]
        device = m[0].device
        for name, xs, ns, dt in (("m", m, numels, torch.float32), ("v", v, numels, torch.float32),
                                 ("m8", m8, numels, M8), ("v8", v8, numels, V8),
                                 ("m8_scale", m8_scale, [scale_count(n) for n in numels], SCALE8),
                                 ("v8_scale", v8_scale, [scale_count(n) for n in numels], SCALE8)):
            _check_list(name, xs, ns, (dt,), device)
        self.stream, self.device = stream, device
        self._keep = (m, v, m8, m8_scale, v8, v8_scale)
        self._list = BoundList(numels, None, 1, B.ZERO_BF16, B.ZERO_NO_OUT, device)
        used_on(stream, [self._list.workspace], *self._keep)
        with _device(device.index):
            self._list.bind(self._s(), m=m, v=v, m8=m8, m8_scale=m8_scale, v8=v8, v8_scale=v8_scale)
        lib = B.lib()
        self._encode, self._decode, self._M = lib.zero_multi_encode8, lib.zero_multi_decode8, self._list.M.handle
        self._index, self._several = device.index, torch.cuda.device_count() > 1

    def _s(self):
        return self.stream if self.stream is not None else torch.cuda.current_stream(self.device)

    def encode(self) -> None:
        if self._several and _current_device() != self._index:
            with _device(self._index):
                return self.encode()
        status = self._encode(self._M, _raw_stream(self._index) if self.stream is None else self.stream.cuda_stream)
        if status:
            B._check(status)

    def decode(self) -> None:
        if self._several and _current_device() != self._index:
            with _device(self._index):
                return self.decode()
        status = self._decode(self._M, _raw_stream(self._index) if self.stream is None else self.stream.cuda_stream)
        if status:
            B._check(status)

    def check(self) -> None:
        """Wait for the calls so far; RuntimeError if one of their kernels reported an error."""
        with _device(self._index):
            bits = B.zero_multi_device_error(self._list.M)
        if bits:
            raise RuntimeError("8-bit states: a codec kernel gave up waiting (error bits %d)" % bits)

    def report(self, state: torch.Tensor) -> None:
        """Add the errors of the calls so far to a device step state's, without waiting."""
        at = B.zero_step_state.error.offset
        with torch.cuda.stream(self._s()):
            state[at:at + 4].view(torch.int32).bitwise_or_(self._list.error_word())


class MultiAdamW:
    """AdamW for the fp32 parameters ``master`` (a list of contiguous CUDA
    tensors, any sizes) from the gradients ``grads`` (bf16, fp16 or fp32), with
    16-bit copies of the updated parameters in ``out16`` if given.

    ``state_bits`` 32 or 8; the states are allocated as zeros unless ``m`` and
    ``v`` (and, for 8 bits, ``m_scale`` and ``v_scale``) are given.  ``groups``
    are hyperparameter groups (one beta1, beta2 for all of them: those live in
    the step state), ``group_of_tensor`` says which a tensor is in.
    ``decide``: compute the global norm first, clip to ``max_norm`` (> 0) and
    skip the step on overflow; by default when there is a ``max_norm`` or a
    loss scale.  ``seed`` seeds the stochastic rounding of 8-bit states.
    ``master`` None makes an object for :meth:`grad_norm` alone.

    The library reads and writes the tensors in place; they must stay
    allocated, and gradients that move are passed to :meth:`rebind_grads`.
    Learning rates of later steps: ``opt.hp[group].lr = x``."""

    def __init__(self, master: Optional[Sequence[torch.Tensor]], grads: Sequence[torch.Tensor],
                 out16: Optional[Sequence[torch.Tensor]] = None, *, state_bits: int = 32, m=None, v=None,
                 m_scale=None, v_scale=None, groups: Sequence[AdamW] = (AdamW(),),
                 group_of_tensor: Optional[Sequence[int]] = None, max_norm: float = 0.0, loss_scale: float = 1.0,
                 dynamic_scale: bool = False, growth_interval: int = 2000, decide: Optional[bool] = None,
                 seed: int = 0, stream: Optional[torch.cuda.Stream] = None):
        if not len(grads):
            raise ValueError("no tensors")
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        if len({(g.beta1, g.beta2) for g in groups}) != 1:
            raise ValueError("all groups share beta1 and beta2")
        self.numels = [g.numel() for g in grads]
        self.device = grads[0].device
        self.stream = stream
        _check_list("grads", grads, self.numels, tuple(_GRAD), self.device)
        if master is not None:
            _check_list("master", master, self.numels, (torch.float32,), self.device)
        if out16 is not None:
            _check_list("out16", out16, self.numels, tuple(_PARAM), self.device)
        no_scaler = not dynamic_scale and loss_scale == 1.0
        self.decide = (max_norm > 0 or not no_scaler) if decide is None else bool(decide)
        if not self.decide and (max_norm > 0 or dynamic_scale):
            raise ValueError("a step without the norm cannot clip or skip")
        self._decided = False        # grad_norm was called since the last update
        self.state_bits, self.max_norm, self.seed = state_bits, float(max_norm), int(seed)
        self.beta1, self.beta2 = groups[0].beta1, groups[0].beta2
        self._hp = (B.zero_adamw_hp * len(groups))(*[B.zero_adamw_hp(lr=g.lr, eps=g.eps, weight_decay=g.weight_decay)
                                                    for g in groups])
        self.master, self.grads, self.out16 = master, grads, out16
        self._states(m, v, m_scale, v_scale)
        self._list = BoundList(self.numels, group_of_tensor, len(groups), _GRAD[grads[0].dtype],
                           _PARAM[out16[0].dtype] if out16 is not None else B.ZERO_NO_OUT, self.device)
        self.info = self._list.info
        self.state = torch.zeros(ctypes.sizeof(B.zero_step_state), dtype=torch.uint8, device=self.device)
        # the calls' arguments that do not change between steps, converted once: a short step costs the
        # host a few microseconds, most of them spent on arguments otherwise
        lib, eight = B.lib(), state_bits == 8
        self._grad_norm, self._adamw = lib.zero_multi_grad_norm, lib.zero_multi_adamw8 if eight else lib.zero_multi_adamw
        self._M = self._list.M.handle
        self._index, self._several = self.device.index, torch.cuda.device_count() > 1
        self._st = ctypes.c_void_p(self.state.data_ptr())
        used_on(stream, [self._list.workspace, self.state], grads, master, out16, self.m, self.v, self.m_scale, self.v_scale)
        self._bind()
        with _device(self._index):
            B.zero_state_init(self.state, self.beta1, self.beta2, loss_scale, dynamic_scale, growth_interval, self._s())

    def _s(self):
        return self.stream if self.stream is not None else torch.cuda.current_stream(self.device)

    @property
    def hp(self):
        """The groups' hyperparameters (``hp[g].lr``, ``.eps``,
        ``.weight_decay``), read at every step."""
        return self._hp

    def _norm(self):
        if self._several and _current_device() != self._index:
            with _device(self._index):
                return self._norm()
        status = self._grad_norm(self._M, self.max_norm, self._st, self._handle())
        if status:
            B._check(status)

    def _update(self, flags):
        if self._several and _current_device() != self._index:
            with _device(self._index):
                return self._update(flags)
        seed = (self.seed & 0xFFFFFFFF,) if self.state_bits == 8 else ()
        status = self._adamw(self._M, self._hp, flags, *seed, self._st, self._handle())
        if status:
            B._check(status)

    def _handle(self) -> int:
        return _raw_stream(self._index) if self.stream is None else self.stream.cuda_stream

    def _states(self, m, v, m_scale, v_scale):
        eight = self.state_bits == 8
        given = [x is not None for x in ((m, v, m_scale, v_scale) if eight else (m, v))]
        if any(given) != all(given) or (not eight and (m_scale is not None or v_scale is not None)):
            raise ValueError("states are given together: m and v%s" % (", m_scale and v_scale" if eight else ""))
        scales = [scale_count(n) for n in self.numels]
        if self.master is None and not any(given):
            m = v = m_scale = v_scale = None
        elif not any(given):
            m, v = (_slices(self.numels, dt, self.device) for dt in ((M8, V8) if eight else (torch.float32,) * 2))
            if eight:
                m_scale, v_scale = (_slices(scales, SCALE8, self.device) for _ in range(2))
        else:
            _check_list("m", m, self.numels, (M8 if eight else torch.float32,), self.device)
            _check_list("v", v, self.numels, (V8 if eight else torch.float32,), self.device)
            if eight:
                _check_list("m_scale", m_scale, scales, (SCALE8,), self.device)
                _check_list("v_scale", v_scale, scales, (SCALE8,), self.device)
        self.m, self.v, self.m_scale, self.v_scale = m, v, m_scale, v_scale

    def _bind(self):
        if self.state_bits == 8:
            states = dict(m8=self.m, v8=self.v, m8_scale=self.m_scale, v8_scale=self.v_scale)
        else:
            states = dict(m=self.m, v=self.v)
        with _device(self._index):
            self._list.bind(self._s(), grads=self.grads, master=self.master, param16=self.out16, **states)

    def rebind_grads(self, grads: Sequence[torch.Tensor]) -> None:
        """Take the gradients from other tensors from the next call on."""
        _check_list("grads", grads, self.numels, (self.grads[0].dtype,), self.device)
        used_on(self.stream, grads)
        self.grads = grads
        self._bind()

    # -- the step ------------------------------------------------------------------
    def grad_norm(self) -> None:
        """The global norm and the step decision alone (one launch)."""
        self._norm()
        self._decided = True

    def update(self, flags: Optional[int] = None) -> None:
        """The update alone (one launch): of the step that ``grad_norm`` has
        decided (``ZERO_MULTI_DECIDED``), or of one without a decision
        (``ZERO_MULTI_ADVANCE``), which is the default for an object with
        ``decide=False`` unless ``grad_norm`` was called since its last update."""
        if flags is None:
            flags = B.ZERO_MULTI_DECIDED if self.decide or self._decided else B.ZERO_MULTI_ADVANCE
        self._update(flags)
        self._decided = False

    def step(self) -> None:
        if self.decide:
            self._norm()
            self._update(B.ZERO_MULTI_DECIDED)
        else:
            self._update(B.ZERO_MULTI_ADVANCE)
            self._decided = False

    def capture(self) -> torch.cuda.CUDAGraph:
        """Record one step into a CUDA graph; replaying it runs one step, with
        the hyperparameters of the recording and the gradients of the last
        :meth:`rebind_grads`.  Replays and the object's other calls are
        ordered like any work: on one stream, or by waits.  The object and its
        tensors must live as long as the graph."""
        g = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream(self.device)
        side.wait_stream(torch.cuda.current_stream(self.device))
        side.wait_stream(self._s())
        old = self.stream
        try:
            self.stream = side
            with torch.cuda.graph(g, stream=side):
                self.step()
        finally:
            self.stream = old
        torch.cuda.current_stream(self.device).wait_stream(side)
        return g

    # -- states ----------------------------------------------------------------------
    def _codec(self, m, v) -> StateCodec8:
        return StateCodec8(m, v, self.m, self.m_scale, self.v, self.v_scale, self.stream)

    def states32(self):
        """(m, v) as lists of new fp32 tensors, e.g. for a checkpoint that an
        optimizer with states of either width can resume from.  An error of
        the decoding kernel shows in ``read_state()["error"]``."""
        cur = torch.cuda.current_stream(self.device)
        if self.state_bits == 32:
            cur.wait_stream(self._s())
            copies = [x.clone() for x in self.m], [x.clone() for x in self.v]
            self._s().wait_stream(cur)       # the next step, on a stream of its own
            return copies
        m, v = (_slices(self.numels, torch.float32, self.device) for _ in range(2))
        codec = self._codec(m, v)
        codec.decode()
        codec.report(self.state)
        cur.wait_stream(self._s())
        return m, v

    def load_states(self, m: Sequence[torch.Tensor], v: Sequence[torch.Tensor]) -> None:
        """Take the states from fp32 tensors (nearest 8-bit values)."""
        if self.state_bits == 32:
            for name, src in (("m", m), ("v", v)):
                _check_list(name, src, self.numels, (torch.float32,), self.device)
            cur = torch.cuda.current_stream(self.device)
            cur.wait_stream(self._s())       # a step under way on a stream of its own
            for src, dst in ((m, self.m), (v, self.v)):
                for a, b in zip(src, dst):
                    b.copy_(a)
            self._s().wait_stream(cur)
        else:
            codec = self._codec(m, v)
            codec.encode()
            codec.report(self.state)
            # the codec's workspace, and the caller's m and v, may be freed after this on the current stream
            torch.cuda.current_stream(self.device).wait_stream(self._s())

    def resume_at(self, t: int) -> None:
        """Set the number of applied steps (bias corrections go by it), as
        after ``t`` steps of an earlier run."""
        if t < 0:
            raise ValueError("t must be >= 0")
        self._s().synchronize()
        st = B.zero_step_state.from_buffer_copy(self.state.cpu().numpy().tobytes())
        st.t, st.beta1_pow, st.beta2_pow = t, 1.0, 1.0
        for _ in range(t):           # t successive products, as the steps form them
            st.beta1_pow *= self.beta1
            st.beta2_pow *= self.beta2
        self.state.copy_(torch.frombuffer(bytearray(bytes(st)), dtype=torch.uint8))
        self._s().wait_stream(torch.cuda.current_stream(self.device))

    def state_fields(self) -> dict:
        """Fields of the device step state as one-element device views, to be
        used without a copy to the host (``read_state`` makes one)."""
        at = {n: getattr(B.zero_step_state, n).offset for n, _ in B.zero_step_state._fields_}
        kinds = {"grad_norm": torch.float64, "loss_scale": torch.float32, "clip_coef": torch.float32, "t": torch.int32,
                 "skipped": torch.int32, "overflow": torch.int32, "apply": torch.int32}
        return {n: self.state[at[n]:at[n] + torch.empty(0, dtype=dt).element_size()].view(dt) for n, dt in kinds.items()}

    def read_state(self) -> dict:
        return read_step_state(self.state)
