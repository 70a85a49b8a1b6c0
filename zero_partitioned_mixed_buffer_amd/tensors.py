"""Adam/AdamW over a list of tensors, with states in 32 or in 8 bits.

Holds the list's states, control block and workspace (allocated with torch)
and forwards each step to the library: zero_tensors_grad_norm where the
gradients are checked or clipped, then zero_tensors_adam_step.  Nothing here
synchronises with the device but the constructor, set_grads(), set_step(),
control() and the checkpoint calls.
"""
from __future__ import annotations

import ctypes as C
from typing import Optional, Sequence

from . import binding as B

_ALIGN = 64  # elements between the starts a state may have in its buffer


class TensorAdam:
    """``masters``: float32 tensors, stepped in place.  ``grads``: their
    gradients, all float32, float16 or bfloat16.  ``params``: float16 or
    bfloat16 copies of the weights that each step writes, or None.

    The states lie in one buffer each (``exp_avg``, ``exp_avg_sq``; with
    state_bits=8 also ``avg_scale`` and ``sq_scale``), tensor i from element
    state_offs[i], a multiple of 64, with zeros in the gaps.  With 8 bits
    ``exp_avg_sq`` holds the variance's root, under stochastic rounding for a
    beta2 of at most 0.9999 (above it variances drift low).  Fill them in
    place.

    The list holds the tensors' addresses.  Gradients that autograd makes anew
    (after zero_grad() with its default, set_to_none=True) are others than
    those it was given: either zero_grad(set_to_none=False) keeps the tensors,
    or set_grads() names the new ones after each backward pass.  Without
    either, steps go on with the old gradients.

    check_finite (default) takes a pass over the gradients first and skips
    the step if any is inf or NaN; max_grad_norm > 0 (clipping) and
    scale_interval > 0 (dynamic loss scaling, from ``loss_scale``) need it.

    Hyperparameters are ``hp``'s fields and may change between steps, as may
    ``loss_scale`` (a step captured in a graph keeps those it was captured
    with).  Lists that share one norm, or ranks that hold parts of the
    parameters, take it apart from the step: grad_norm() on each, then the
    sums added and the flags OR-ed, then step(norm=...).

    Masters and params that require gradients (when the list is made) count
    each step as torch's in-place operations do, so that a backward pass
    through a graph made before it raises; aliases that do not (p.data,
    p.detach()) and replays of a captured step are not counted.
    """

    def __init__(self, masters: Sequence, grads: Sequence, params: Optional[Sequence] = None,
                 flat_offs: Optional[Sequence[int]] = None, state_bits: int = 32, lr=1e-3, beta1=0.9, beta2=0.999,
                 eps=1e-8, weight_decay=0.0, max_grad_norm=0.0, check_finite=True, scale_interval=0,
                 scale_growth=2.0, scale_backoff=0.5, loss_scale=1.0, rounding="stochastic", seed=0):
        import torch
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits: {state_bits}, expected 8 or 32")
        if not len(masters):
            raise ValueError("an empty list of tensors")
        if not check_finite and (max_grad_norm > 0 or scale_interval > 0):
            raise ValueError("clipping and dynamic loss scaling need check_finite")
        B._rounding(rounding)
        self.device = masters[0].device
        if self.device.type != "cuda":
            raise ValueError("masters: must be device tensors")
        self.masters, self.grads = list(masters), list(grads)
        self.params = list(params) if params is not None else None
        self.flat_offs = None if flat_offs is None else [int(x) for x in flat_offs]
        self.state_bits = state_bits
        self.numels = [int(t.numel()) for t in self.masters]
        self.state_offs, total = [], 0
        for n in self.numels:
            self.state_offs.append(total)
            total += -(-n // _ALIGN) * _ALIGN
        dev = self.device
        with torch.cuda.device(dev):
            if state_bits == 8:
                def byte(n, x, kind):
                    return torch.full((n,), x, dtype=torch.uint8, device=dev).view(kind)
                self.exp_avg, self.exp_avg_sq = (byte(total, 0, torch.float8_e4m3fn) for _ in range(2))
                # the scale byte of an encoded block of zeros
                self.avg_scale, self.sq_scale = (byte(total // B.MX8_BLOCK, 1, torch.float8_e8m0fnu)
                                                 for _ in range(2))
            else:
                self.exp_avg, self.exp_avg_sq = (torch.zeros(total, dtype=torch.float32, device=dev)
                                                 for _ in range(2))
                self.avg_scale = self.sq_scale = None
            self.ctl = torch.frombuffer(bytearray(B.ctl_init_bytes(loss_scale)), dtype=torch.uint8).to(dev)
            self.workspace = torch.zeros(B.workspace_bytes(), dtype=torch.uint8, device=dev)
            self.overflow = torch.zeros(1, dtype=torch.int32, device=dev)
            self.sumsq = torch.zeros(1, dtype=torch.float64, device=dev)
        self.hp = B.adam_hp(lr, beta1, beta2, eps, weight_decay, max_grad_norm, scale_interval, scale_growth,
                            scale_backoff)
        self.loss_scale = float(loss_scale)
        self.check_finite = bool(check_finite)
        self.rounding = rounding if state_bits == 8 else "nearest"
        self.seed = int(seed) & (2**64 - 1)
        self._plan()
        # the buffers are filled before a step on any stream
        torch.cuda.current_stream(dev).synchronize()

    def _tensor_list(self, grads, flat_offs=None):
        import torch
        mx = self.state_bits == 8
        with torch.cuda.device(self.device):
            gtype, ptrs, numels = B._grad_column(grads)
            if numels != self.numels:
                raise ValueError("gradients: the sizes of the master weights expected")
            columns = {"grad": ptrs, "master": B._column(self.masters, numels, ("float32",), "masters")[1]}
            ptype, keep = B.TYPE_NONE, [grads, self.masters, self.exp_avg, self.exp_avg_sq]
            if self.params is not None:
                name, columns["param"] = B._column(self.params, numels, ("float16", "bfloat16"), "params")
                ptype = B._LIST_TYPES[name]
                keep.append(self.params)
            B._on_current([grads, self.masters, self.params or ()])
            for name, flat, per in (("exp_avg", self.exp_avg, 1), ("exp_avg_sq", self.exp_avg_sq, 1),
                                    ("avg_scale", self.avg_scale, B.MX8_BLOCK),
                                    ("sq_scale", self.sq_scale, B.MX8_BLOCK)):
                if flat is not None:
                    base, size = flat.data_ptr(), flat.element_size()
                    columns[name] = [base + o // per * size for o in self.state_offs]
                    keep.append(flat)
            return B._plan_list(numels, columns, gtype, ptype, B.TYPE_MX8 if mx else B.TYPE_F32,
                                self.flat_offs if flat_offs is None else flat_offs, keep,
                                (*self.masters, *(self.params or ())))

    def _plan(self):
        self.list = self._tensor_list(self.grads)
        # the calls' fixed arguments; every buffer is this object's own
        table = None if self.list.table is None else self.list.table.data_ptr()
        self._head = (self.list.ref, table)
        self._checks = (self.overflow.data_ptr(), self.sumsq.data_ptr())
        self._ctl, self._ws = self.ctl.data_ptr(), self.workspace.data_ptr()

    def _offs(self):
        """The tensors' first random counters (by default packed in list order)."""
        if self.flat_offs is not None:
            return self.flat_offs
        at, offs = 0, []
        for n in self.numels:
            offs.append(at)
            at += n
        return offs

    def set_grads(self, grads: Sequence):
        """Other gradient tensors of the same sizes and dtype, from the next
        step on the current stream (steps under way on other streams have to
        have ended).  The list's table is rewritten in place, so that steps
        captured in a graph read the new tensors too."""
        import torch
        grads = list(grads)
        new = self._tensor_list(grads)
        if new.info.grad_type != self.list.info.grad_type:
            raise ValueError(f"gradients: dtype {grads[0].dtype}, but the list was planned with {self.grads[0].dtype}")
        with torch.cuda.device(self.device):
            if new.table is not None:
                self.list.table.copy_(new.table)
        self.list.tensors, self.grads = new.tensors, grads

    def grad_norm(self, stream=None):
        """The gradients' sum of squares (``sumsq``, unscaled) and inf/NaN flag
        (``overflow``), device tensors of this object; returns both."""
        if B._current_device() != self.device.index:
            import torch
            with torch.cuda.device(self.device):
                return self.grad_norm(stream)
        dyn = self._ctl if self.hp.scale_interval > 0 else None
        B._check(B.lib().zero_tensors_grad_norm(*self._head, self.loss_scale, dyn, self.overflow.data_ptr(),
                                                self.sumsq.data_ptr(), self._ws, B._stream(stream)),
                 "zero_tensors_grad_norm")
        return self.overflow, self.sumsq

    def step(self, stream=None, norm=None):
        """One step on what the gradient tensors hold, scaled by ``loss_scale``
        (with dynamic scaling by the control block's).  ``norm``: the (flag,
        sum of squares) device tensors to go by, int32 and float64, where they
        were taken elsewhere; no pass over the gradients is made then."""
        if B._current_device() != self.device.index:
            import torch
            with torch.cuda.device(self.device):
                return self.step(stream, norm)
        if norm is not None:
            overflow, sumsq = norm
            B._check_operand(overflow, 1, ("int32",), "overflow flag", self.device.index)
            B._check_operand(sumsq, 1, ("float64",), "sum of squares", self.device.index)
            checks = (B._ptr(overflow), B._ptr(sumsq))
        elif self.check_finite:
            self.grad_norm(stream)
            checks = self._checks
        else:
            checks = (None, None)
        B._check(B.lib().zero_tensors_adam_step(*self._head, C.byref(self.hp), self.loss_scale, self._ctl, *checks,
                                                B.ROUNDING[self.rounding], self.seed, self._ws, B._stream(stream)),
                 "zero_tensors_adam_step")
        self.list.count_write()

    def _wait(self):
        """Every stream of the device: a step may run on any of them."""
        import torch
        torch.cuda.synchronize(self.device)

    def control(self) -> dict:
        """Reads the device control block (synchronises with the device)."""
        self._wait()
        return B.ctl_from_bytes(bytes(self.ctl.cpu().numpy().tobytes()))

    def set_step(self, t: int):
        """Makes ``t`` the number of steps taken so far (beta powers as t
        successive products).  Synchronises with the device."""
        if t < 0:
            raise ValueError("a negative step count")
        c = self.control()
        c["t"], c["beta1_pow"], c["beta2_pow"] = int(t), 1.0, 1.0
        for _ in range(int(t)):
            c["beta1_pow"] *= self.hp.beta1
            c["beta2_pow"] *= self.hp.beta2
        self._write_control(c)

    def _write_control(self, fields: dict):
        import torch
        self.ctl.copy_(torch.frombuffer(bytearray(B.ctl_to_bytes(fields)), dtype=torch.uint8))

    # ------------------------------------------------------------ checkpoint
    def state_dict(self) -> dict:
        """Host copies of the weights, states (codes and scale bytes as uint8
        for 8 bits) and the control block; for 8 bits also what the random
        words depend on (seed, rounding and flat_offs).  Synchronises with
        the device."""
        import numpy as np
        import torch
        self._wait()

        def host(x):
            return (x if x.dtype == torch.float32 else x.view(torch.uint8)).cpu().numpy()

        out = {"numels": np.asarray(self.numels, dtype=np.int64),
               "master": np.concatenate([m.detach().reshape(-1).cpu().numpy() for m in self.masters]),
               "exp_avg": host(self.exp_avg), "exp_avg_sq": host(self.exp_avg_sq),
               "ctl": np.frombuffer(self.ctl.cpu().numpy().tobytes(), dtype=np.uint8).copy()}
        if self.state_bits == 8:
            out["avg_scale"], out["sq_scale"] = host(self.avg_scale), host(self.sq_scale)
            out["seed"], out["rounding"] = np.uint64(self.seed), np.asarray(self.rounding)
            out["flat_offs"] = np.asarray(self._offs(), dtype=np.int64)
        return out

    def load_state_dict(self, sd: dict):
        """Restores a state_dict of a list of the same sizes.  Of the same
        state_bits, under the same hyperparameters, it resumes exactly: 8-bit
        states bring their seed, rounding and flat_offs along (a step captured
        in a graph keeps the seed and rounding it was captured with).  States
        of the other width are encoded (to nearest) or decoded; a variance
        that float32 does not hold (a gradient above 1e19 was met) is then
        taken as its largest value and its momentum cut with it, so that the
        weight's next updates keep their size, or stay below lr where that
        size is lost too (an infinite 32-bit variance).  The 16-bit copies
        are written anew.  Synchronises with the device."""
        import numpy as np
        import torch
        if [int(x) for x in np.asarray(sd["numels"])] != self.numels:
            raise ValueError("numels: the state_dict is of a list of other sizes")
        raw = np.asarray(sd["ctl"], dtype=np.uint8).tobytes()
        if len(raw) != B.CTL_BYTES:
            raise ValueError(f"control block: expected {B.CTL_BYTES} bytes, got {len(raw)}")
        total = self.exp_avg.numel()
        mx = "avg_scale" in sd
        want = {"master": (np.float32, sum(self.numels))}
        for k in ("exp_avg", "exp_avg_sq"):
            want[k] = (np.uint8 if mx else np.float32, total)
        if mx:
            want["avg_scale"] = want["sq_scale"] = (np.uint8, total // B.MX8_BLOCK)
        for k, (kind, n) in want.items():
            a = np.asarray(sd[k])
            if a.dtype != kind or a.shape != (n,):
                raise ValueError(f"{k}: expected {np.dtype(kind).name}[{n}], got {a.dtype}{list(a.shape)}")
        words = None
        if mx and self.state_bits == 8 and "seed" in sd:
            words = (int(np.asarray(sd["seed"])), str(np.asarray(sd["rounding"])),
                     [int(x) for x in np.asarray(sd["flat_offs"])])
            B._rounding(words[1])
            # planned before anything is written: wrong offsets are refused
            new = self._tensor_list(self.grads, words[2]) if words[2] != self._offs() else None
        self._wait()
        with torch.cuda.device(self.device):
            arr = {k: torch.from_numpy(np.ascontiguousarray(sd[k])).to(self.device) for k in want}
            at = 0
            for i, (m, n) in enumerate(zip(self.masters, self.numels)):
                m.detach().view(-1).copy_(arr["master"][at:at + n])
                if self.params is not None:
                    self.params[i].detach().view(-1).copy_(m.detach().view(-1))
                at += n
            if not mx and self.state_bits == 8:
                self._cut_variances(arr["exp_avg"], arr["exp_avg_sq"])
            for k, scale, root in (("exp_avg", "avg_scale", False), ("exp_avg_sq", "sq_scale", True)):
                mine = getattr(self, k)
                if mx and self.state_bits == 8:
                    mine.view(torch.uint8).copy_(arr[k])
                    getattr(self, scale).view(torch.uint8).copy_(arr[scale])
                elif mx:
                    B.mx8_decode(arr[k], arr[scale], mine, root=root)
                elif self.state_bits == 8:
                    B.mx8_encode(arr[k], mine, getattr(self, scale), root=root, rounding="nearest")
                else:
                    mine.copy_(arr[k])
            if mx and self.state_bits == 32 and bool(self.exp_avg_sq.isinf().any()):
                root = torch.empty_like(self.exp_avg_sq)
                B.mx8_decode(arr["exp_avg_sq"], arr["sq_scale"], root)
                self._cut_variances(self.exp_avg, self.exp_avg_sq, root)
            if words is not None:
                self.seed, self.rounding = words[0] & (2**64 - 1), words[1]
                if new is not None:
                    self.flat_offs, self.list.tensors = words[2], new.tensors
                    if new.table is not None:
                        self.list.table.copy_(new.table)
            self._write_control(B.ctl_from_bytes(raw))
            self._wait()

    @staticmethod
    def _cut_variances(m, v, root=None):
        """Variances past float32's range (inf) become its largest value, and
        their momenta shrink in the same proportion to the variance's root
        2^64; where the root is not known, to no more than that."""
        import torch
        past = v.isinf()
        m.copy_(torch.where(past, m.clamp(-2.0 ** 64, 2.0 ** 64) if root is None else m * (2.0 ** 64 / root), m))
        v.masked_fill_(past, torch.finfo(torch.float32).max)

    def save(self, path: str):
        """Writes state_dict() to a .npz file (plain arrays, no pickles)."""
        import numpy as np
        np.savez(path, **self.state_dict())

    def load(self, path: str):
        """Restores a file written by save() (loaded without pickles)."""
        import numpy as np
        with np.load(path, allow_pickle=False) as z:
            self.load_state_dict({k: z[k] for k in z.files})
