"""Rotary positions and the page planner: torch-facing wrappers over the libspectra C ABI."""
from __future__ import annotations

import ctypes

from ._lib import ROPE_SCALINGS, SPECTRA_BF16, SPECTRA_F32, HeadsDesc, RopeDesc, check, lib
from .codec import _check_tensor, _fresh, _on, _same_device, _torch


class Rope:
    """A rotary embedding: base, rotated dimensions, pairing and scaling of the frequencies.

    theta: base; rot_dim: rotated leading dimensions of a head (0: all); interleaved: pairs (2i, 2i+1) instead of
    (i, i + rot_dim/2); scaling: "none", "linear", "ntk", "llama3" or "yarn" with ``factor``, and for the last two
    ``original_len`` and the band ``low`` < ``high``; magnitude: factor on cosine and sine (0: the scaling's own).
    The formulas are in ``include/spectra.h``.
    """

    def __init__(self, theta: float = 10000.0, rot_dim: int = 0, interleaved: bool = False, scaling: str = "none",
                 factor: float = 1.0, low: float = 1.0, high: float = 4.0, original_len: int = 0,
                 magnitude: float = 0.0):
        if scaling not in ROPE_SCALINGS:
            raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}")
        self.desc = RopeDesc(float(theta), float(factor), float(low), float(high), float(magnitude),
                             ROPE_SCALINGS[scaling], int(original_len), int(rot_dim), int(bool(interleaved)))

    def frequencies(self, d_head: int):
        """(radians per position of each pair, the factor on cosine and sine), as the kernels use them."""
        import numpy as np
        rot = self.desc.rot_dim or int(d_head)
        freq = np.zeros(max(rot, 2) // 2, np.float64)
        mag = ctypes.c_double()
        check(lib.spectra_rope_frequencies(ctypes.byref(self.desc), int(d_head), None, None),
              "spectra_rope_frequencies")
        check(lib.spectra_rope_frequencies(ctypes.byref(self.desc), int(d_head), freq.ctypes.data, ctypes.byref(mag)),
              "spectra_rope_frequencies")
        return freq, mag.value

    def apply(self, positions, q, k=None, q_out=None, k_out=None, inverse: bool = False, stream=None):
        """Rotated (q, k) of [tokens][heads][d_head] tensors (fp32 or bf16, any token and head strides), in one
        launch.  Outputs may be the inputs, and overlap nothing else.  Rows with a negative position are left out:
        fresh outputs hold a copy of the input there.  ``inverse`` takes the rotation back.  The call is not recorded
        for autograd: fresh outputs need no gradient, and a given output that needs one is refused while gradients are
        recorded.  With magnitude 1 the inputs' gradients are ``apply`` of the outputs' with ``inverse`` flipped."""
        torch = _torch()
        if q.dtype is torch.bfloat16:
            dt = SPECTRA_BF16
        elif q.dtype is torch.float32:
            dt = SPECTRA_F32
        else:
            raise TypeError("q must be bfloat16 or float32")
        if q.dim() != 3:
            raise ValueError("q must be [tokens][heads][d_head]")
        T, _, d = q.shape
        _check_tensor("positions", positions, torch.int32, (T,))
        _same_device(q, positions=positions)
        if k is None and k_out is not None:
            raise ValueError("k_out without k")
        with _on(q, stream) as st:
            q_in, q_o, q_out = _pair("q", q, q_out, T, d, q, st)
            k_in = k_o = None
            if k is not None:
                k_in, k_o, k_out = _pair("k", k, k_out, T, d, q, st)
            check(lib.spectra_rope_apply(self.desc, dt, d, positions.data_ptr(), T, q_in, q_o, k_in, k_o,
                                         1 if inverse else 0, st.raw), "spectra_rope_apply")
        return q_out, k_out


def _heads(name, t, n_heads):
    step = t.stride()
    if step[2] != 1 and t.numel():
        raise ValueError(f"{name} needs contiguous head vectors")
    return HeadsDesc(t.data_ptr(), step[0], step[1], n_heads)


def _pair(name, x, out, T, d, like, st):
    """Descriptors of an input and its output, and the output (fresh if None)."""
    shape = x.shape
    if len(shape) != 3 or shape[0] != T or shape[2] != d:
        raise ValueError(f"{name} must be [tokens][heads][d_head], alike in tokens and d_head")
    index = like.get_device()
    if x.dtype is not like.dtype or x.get_device() != index:
        raise TypeError(f"{name} must have q's type and device")
    n = shape[1]
    given = _heads(name, x, n)
    if out is None:
        out = _copied(x, st)
        return given, _heads(name + "_out", out, n), out
    if out is not x and (out.shape != shape or out.dtype is not like.dtype or out.get_device() != index):
        raise ValueError(f"{name}_out must be like {name}")
    torch = _torch()
    if out.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name}_out needs a gradient, which the call does not record")
    torch._C._increment_version((out,))  # (a graph may hold it for its backward pass)
    return given, given if out is x else _heads(name + "_out", out, n), out


def _copied(x, st):
    """A copy of `x` in one row of vectors, made in the call's stream and unknown to autograd."""
    torch = _torch()
    x = x.detach()
    if st.side is None:
        return x.clone(memory_format=torch.contiguous_format)
    out = _fresh(torch.empty(x.shape, dtype=x.dtype, device=x.device), st)
    with torch.cuda.stream(st.side):
        out.copy_(x)
    return out


class AppendPlan:
    """Output tensors of ``PagePlanner.plan_append`` for up to ``max_tokens`` tokens of ``batch`` sequences.

    Other tensors of the same type, size and device may be put in their place."""

    def __init__(self, max_tokens: int, batch: int, device="cuda"):
        torch = _torch()
        self._max_tokens, self._batch = int(max_tokens), int(batch)
        T, self._tensors = self._max_tokens, {}
        for name, n, dtype in (("seq_ids", T, torch.int32), ("positions", T, torch.int32), ("slots", T, torch.int64),
                               ("offsets", self._batch + 1, torch.int32)):
            self._tensors[name] = torch.empty(n, dtype=dtype, device=device)

    max_tokens = property(lambda self: self._max_tokens)
    batch = property(lambda self: self._batch)

    def _put(self, name, t):
        old = self._tensors[name]
        if t.dtype != old.dtype:
            raise TypeError(f"{name} must be {old.dtype}")
        if t.shape != old.shape or not t.is_contiguous() or t.device != old.device:
            raise ValueError(f"{name} must be contiguous, of shape {tuple(old.shape)} and on {old.device}")
        self._tensors[name] = t

    seq_ids = property(lambda self: self._tensors["seq_ids"], lambda self, t: self._put("seq_ids", t))
    positions = property(lambda self: self._tensors["positions"], lambda self, t: self._put("positions", t))
    slots = property(lambda self: self._tensors["slots"], lambda self, t: self._put("slots", t))
    offsets = property(lambda self: self._tensors["offsets"], lambda self, t: self._put("offsets", t))


class PagePlanner:
    """Gives sequences their cache pages on the GPU and takes them back.

    The caller keeps a stack of free page ids (``free_pages`` int32 [capacity], ``n_free`` int32 [1]) beside the
    cache's page table and lengths, all on the GPU; one planner serves every layer that shares the table.
    """

    def __init__(self, page_tokens: int, device="cuda"):
        torch = _torch()
        self.page_tokens = int(page_tokens)
        self.device = torch.device(device)
        self._h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            check(lib.spectra_planner_create(self.page_tokens, ctypes.byref(self._h)), "spectra_planner_create")

    def close(self):
        if self._h:
            lib.spectra_planner_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def plan_append(self, page_table, lengths, new_tokens, free_pages, n_free, prefix_pages=None, n_free_out=None,
                    plan=None, max_tokens=None, stream=None) -> AppendPlan:
        """Pages, sequence ids, positions and slots of the next append (``spectra_plan_append``): updates
        ``page_table`` and ``n_free`` (or writes ``n_free_out``) and fills ``plan``; an ``n_free`` above the size of
        ``free_pages`` is an error that ``status`` raises.  Rows of the plan behind the
        last token hold -1; ``Rope.apply`` passes over them, an append takes ``seq_ids[:number of tokens]``."""
        torch = _torch()
        i32 = torch.int32
        B, most = page_table.shape
        _check_tensor("page_table", page_table, i32, (B, most))
        _check_tensor("lengths", lengths, i32, (B,))
        _check_tensor("new_tokens", new_tokens, i32, (B,))
        _check_tensor("free_pages", free_pages, i32, (free_pages.numel(),))
        _check_tensor("n_free", n_free, i32, (1,))
        n_prefix = 0
        if prefix_pages is not None:
            n_prefix = prefix_pages.numel()
            _check_tensor("prefix_pages", prefix_pages, i32, (n_prefix,))
        if n_free_out is None:
            n_free_out = n_free
        else:
            _check_tensor("n_free_out", n_free_out, i32, (1,))
        _same_device(lengths, page_table=page_table, new_tokens=new_tokens, free_pages=free_pages, n_free=n_free,
                     prefix_pages=prefix_pages, n_free_out=n_free_out, plan=None if plan is None else plan.offsets)
        with _on(lengths, stream) as st:
            if plan is None:
                if max_tokens is None:
                    raise ValueError("max_tokens is needed without a plan")
                plan = AppendPlan(max_tokens, B, lengths.device)
                for t in (plan.seq_ids, plan.positions, plan.slots, plan.offsets):
                    _fresh(t, st)
            elif plan.batch != B:
                raise ValueError("the plan was made for another batch")
            check(lib.spectra_plan_append_ex(
                self._h, B, lengths.data_ptr(), new_tokens.data_ptr(), prefix_pages.data_ptr() if n_prefix else None,
                n_prefix, free_pages.data_ptr(), free_pages.numel(), n_free.data_ptr(), n_free_out.data_ptr(),
                page_table.data_ptr(), most, plan.max_tokens, plan.seq_ids.data_ptr(), plan.positions.data_ptr(),
                plan.slots.data_ptr(), plan.offsets.data_ptr(), st.raw), "spectra_plan_append_ex")
        return plan

    def release(self, page_table, lengths, finished, free_pages, n_free, n_prefix: int = 0, stream=None):
        """Gives back the pages of the sequences with ``finished`` (int32) nonzero and empties them."""
        torch = _torch()
        i32 = torch.int32
        B, most = page_table.shape
        _check_tensor("page_table", page_table, i32, (B, most))
        _check_tensor("lengths", lengths, i32, (B,))
        _check_tensor("finished", finished, i32, (B,))
        _check_tensor("free_pages", free_pages, i32, (free_pages.numel(),))
        _check_tensor("n_free", n_free, i32, (1,))
        _same_device(lengths, page_table=page_table, finished=finished, free_pages=free_pages, n_free=n_free)
        with _on(lengths, stream) as st:
            check(lib.spectra_release_pages(self._h, B, finished.data_ptr(), lengths.data_ptr(), int(n_prefix),
                                            page_table.data_ptr(), most, free_pages.data_ptr(), free_pages.numel(),
                                            n_free.data_ptr(), st.raw), "spectra_release_pages")

    def status(self, stream=None):
        """Synchronises the stream; raises what a kernel recorded, and clears it."""
        torch = _torch()
        with torch.cuda.device(self.device):
            raw = int((stream or torch.cuda.current_stream()).cuda_stream)
            check(lib.spectra_planner_status(self._h, raw), "spectra_planner_status")
