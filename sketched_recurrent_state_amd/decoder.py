"""Window cadence of the SketchSSM decode path for one linear-attention layer, and what a layer
has around its recurrence.

``WindowedDecoder`` owns the device buffers of one layer (the state, the
sketch, the W-token window buffer) and sequences the library calls:

* every decode step: the current token goes into its window slot and the
  output is read (from the sketch, or exactly from the full state);
* after the W-th token of a window: one fused update + refresh writes the
  full state once and stores the new sketch, and the window restarts.

This follows the SketchSSM pages (readsearch.ai listing of arXiv 2609.33051,
Abstract: full-state updates once per window with a sketch refresh, sketch
reads in between; agihunt.info summary, "Error control": the sketch's error
never reaches the state). Memory comes from PyTorch; all arithmetic is in the
library's kernels.

``ShortConv`` keeps the last inputs of a layer's short convolution, ``GatedNorm`` the weights of its
output norm; both decoders take them, and then take projections and return normalised outputs.
``SelectiveDecoder`` holds the state of a selective layer (a decay per channel and state).
"""
from __future__ import annotations

import operator
from typing import Optional

import torch

from . import (ConvDims, Dims, IN_BF16, IN_F32, KDA, MAMBA2, NormDims, SKETCH_BF16, SelectiveDims,
               buffer_append, conv_forward, conv_step, full_read_decode_step, gated_norm,
               gated_norm_sizes, rank_offsets, recurrent_decode_step, scan_forward, scan_plan,
               scan_sizes, selective_forward, selective_step, sketch_decode_step, sketch_decode_step_ls,
               sketch_decode_step_ranked, window_update_refresh, window_update_refresh_ls,
               window_update_refresh_ranked, _addr, _row_addr)


def _in_type(in_dtype: int) -> torch.dtype:
    return torch.bfloat16 if in_dtype == IN_BF16 else torch.float32


def _checked_lengths(d, lengths, q):
    """Prompt lengths as Python integers that sum to q's tokens, or the device tensor, which is
    not read back."""
    if isinstance(lengths, torch.Tensor) and lengths.is_cuda:
        if lengths.is_floating_point() or lengths.is_complex() or lengths.numel() != d.batch:
            raise ValueError(f"lengths: {lengths.dtype} {tuple(lengths.shape)}, "
                             f"expected integers ({d.batch},)")
        return lengths
    if hasattr(lengths, "reshape"):  # a tensor or an array: its numbers, of whatever width
        lengths = lengths.reshape(-1).tolist()
    lengths = [operator.index(n) for n in lengths]
    if len(lengths) != d.batch:
        raise ValueError(f"{len(lengths)} lengths for a batch of {d.batch}")
    if min(lengths, default=0) < 0 or sum(lengths) != q.shape[0]:
        raise ValueError(f"lengths sum to {sum(lengths)}, the token arrays hold {q.shape[0]}")
    return lengths


def _plan(lengths, total: int, device) -> torch.Tensor:
    """The plan of a packed batch (checked lengths). Lengths on the device may sum to less than total."""
    if isinstance(lengths, torch.Tensor) and lengths.dtype != torch.int32:
        lengths = lengths.long().clamp(0, total)  # so that the cast cannot wrap
    lengths = torch.as_tensor(lengths, dtype=torch.int32, device=device)
    n = lengths.numel()
    plan = torch.empty(2 * (n + 1) + total // 64 + n, dtype=torch.int32, device=device)
    scan_plan(lengths, total, plan)
    return plan


def _new_rows(lengths):
    """How outputs are made: rows behind the last prompt, if there can be any, are not written, and zero."""
    return torch.zeros if isinstance(lengths, torch.Tensor) else torch.empty


class ShortConv:
    """The short convolution of a layer's inputs (dims.parts of them) for dims.batch sequences.

    weight: fp32 [C, taps], bias: fp32 [C] or None, C the parts' channels one after another
    state:  the last taps - 1 inputs [batch, taps - 1, C] in dims.in_dtype (zeros if None), used in place
    """

    def __init__(self, dims: ConvDims, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                 state: Optional[torch.Tensor] = None):
        self.d, self.weight, self.bias = dims, weight, bias
        self.widths = list(dims.channels[:dims.parts])
        if state is None:
            state = torch.zeros((dims.batch, dims.taps - 1, sum(self.widths)), device=weight.device,
                                dtype=_in_type(dims.in_dtype))
        self.state = state

    def _out(self, make, rows: int):
        return [make((rows, w), device=self.state.device, dtype=self.state.dtype) for w in self.widths]

    def step(self, *xs) -> list:
        """One token of every sequence: the parts' rows [batch][channels], in and out."""
        y = self._out(torch.empty, self.d.batch)
        conv_step(self.d, xs, self.weight, self.bias, self.state, y)
        return y

    def prefill(self, lengths, *xs) -> list:
        """A packed batch of prompts (lengths as in WindowedDecoder.prefill; the parts' rows
        [sum of lengths][channels]): the parts' outputs, and the state continued."""
        lengths = _checked_lengths(self.d, lengths, xs[0])
        with torch.cuda.device_of(self.state):
            return self._prefill(_plan(lengths, xs[0].shape[0], self.state.device), _new_rows(lengths), xs)

    def _prefill(self, plan, make, xs) -> list:
        total = xs[0].shape[0]
        y = self._out(make, total)
        conv_forward(self.d, total, plan, xs, self.weight, self.bias, y, self.state, state_in=self.state)
        return y


class GatedNorm:
    """The norm of a layer's outputs in groups of channels, gated: weight (and bias) fp32
    [groups][width], or [width] with dims.shared."""

    def __init__(self, dims: NormDims, weight: torch.Tensor, bias: Optional[torch.Tensor] = None):
        self.d, self.weight, self.bias = dims, weight, bias

    def check(self, rows: int, gate: Optional[torch.Tensor], device: Optional[int] = None) -> list:
        """Raises where the norm would: a gate for `rows` rows that is missing, not wanted or not such rows,
        weights that are not the dimensions', any of them on another device than `device` (a number, or None). Returns
        the places of the gate and the weights (first byte, and the one behind the last)."""
        if (gate is None) != (self.d.gate == 0):
            raise ValueError("gate: " + ("the norm needs one" if gate is None else "the norm has none"))
        d = self.d
        wide, own, places = d.groups * d.width, d.width if d.shared else d.groups * d.width, []
        if gate is not None:
            tin = _in_type(d.in_dtype)
            at, stride = _row_addr(gate, "gate", (tin,), rows, wide)
            if stride < wide or stride % 8 or stride >= 1 << 26:
                raise ValueError(f"gate: a stride of {stride}, not a multiple of 8 in [{wide}, 2^26)")
            if at % 16:
                raise ValueError("gate: not 16-byte aligned")
            if device is not None and not isinstance(gate, int) and gate.get_device() != device:
                raise ValueError(f"gate: on device {gate.get_device()}, the state is on {device}")
            places.append((at, at + (max(rows - 1, 0) * stride + wide) * tin.itemsize))
        places.append(_place(self.weight, "weight", own, 16, device))
        if self.bias is not None:
            places.append(_place(self.bias, "bias", own, 16, device))
        return places

    def __call__(self, x: torch.Tensor, gate: Optional[torch.Tensor] = None) -> torch.Tensor:
        """x: rows of groups * width channels, whatever its further dimensions; gate: rows of as many: a new tensor of
        x's shape."""
        out = torch.empty(x.shape, device=x.device, dtype=_in_type(self.d.in_dtype))
        gated_norm(self.d, x.shape[0], x, gate, self.weight, self.bias, out)
        return out


def _around(d: Dims, conv: Optional[ShortConv], norm: Optional[GatedNorm]) -> None:
    """Whether a decoder's convolution and norm fit its layer."""
    if conv is not None:
        want = [d.heads * d.d_k, d.heads * d.d_k, d.heads * d.d_v]
        if conv.widths != want or conv.d.batch != d.batch or conv.d.in_dtype != d.in_dtype:
            raise ValueError(f"{conv.d} does not make the queries, keys and values of {d}")
    if norm is not None:  # groups of any channels of a row: heads, runs of heads (Mamba-2), all of them
        if norm.d.groups * norm.d.width != d.heads * d.d_v or norm.d.x_dtype != IN_F32:
            raise ValueError(f"{norm.d} does not take the outputs of {d}")
        gated_norm_sizes(norm.d, 0)  # raises for dimensions that the norm refuses: not after a state is written


_F32 = (torch.float32,)


def _place(x, name: str, count: int, align: int, device: Optional[int]) -> tuple:
    """First byte of a contiguous fp32 argument of `count` elements and the byte behind its last ((0, 0) for None); raises
    where the library would refuse it, or where it is on another device."""
    at = _addr(x, name, _F32, count)
    if at is None:
        return 0, 0
    if at % align:
        raise ValueError(f"{name}: not {align}-byte aligned")
    if device is not None and not isinstance(x, int) and x.get_device() != device:
        raise ValueError(f"{name}: on device {x.get_device()}, the state is on {device}")
    return at, at + 4 * count


def _whole(x: torch.Tensor) -> tuple:
    at = x.data_ptr()
    return at, at + x.numel() * x.element_size()


def _check_around(d: Dims, rows: int, conv, norm, decay, beta, gate, state, *, align=(16, 16), written=(),
                  kept=(), ys=()) -> None:
    """What the recurrence or the norm would refuse of a call's arguments is refused before the convolution or
    the recurrence has written its state: a call that raises for its arguments has done none of its work.
    align: of decay's and beta's addresses; written: what the recurrence writes besides the state; kept: what else
    of the decoder's the caller's outputs ys must not lie over."""
    if norm is None:
        if gate is not None:
            raise ValueError("gate: the decoder has no norm")
        if conv is None:
            return
    device, units = state.get_device(), rows * d.heads
    read = [] if norm is None else norm.check(rows, gate, device)
    own = [_whole(state)]
    if conv is not None:
        if decay is None or (beta is None) != (d.rule == MAMBA2):
            raise ValueError("decay and beta: every rule needs decay, all but Mamba-2 beta")
        read.append(_place(decay, "decay", units * d.d_k if d.rule == KDA else units, align[0], device))
        if beta is not None:
            read.append(_place(beta, "beta", units, align[1], device))
        own.append(_whole(conv.state))
    own += written
    for lo, hi in own:
        for at, end in read:
            if at < hi and lo < end:
                raise ValueError("an array that the call reads overlaps one that it writes")
    for y in ys:
        if y is None:
            continue
        y = _place(y, "y", units * d.d_v, 16, device)
        for at, end in read + own + [_whole(t) for t in kept if t is not None]:
            if at < y[1] and y[0] < end:
                raise ValueError("y overlaps an array that the call reads or that the decoder keeps")
        read.append(y)


def _elsewhere(dec) -> bool:
    """Whether a step of a decoder with a convolution or a norm has to change the current device: the calls of the
    recurrence go to its stream, those of the convolution and the norm to that of their tensors' device."""
    return ((dec.conv is not None or dec.norm is not None)
            and dec.state.get_device() != torch.cuda.current_device())


def _prefill_check(d: Dims, rows: int, conv, norm, decay, beta, gate, state) -> None:
    """_check_around for a packed batch, which asks less of its gates' addresses."""
    if conv is not None:
        scan_sizes(d, rows)  # more tokens than the recurrence takes
    _check_around(d, rows, conv, norm, decay, beta, gate, state, align=(16 if d.rule == KDA else 4, 4))


def _prefill(d: Dims, state: torch.Tensor, lengths, q, k, v, decay, beta, conv=None, norm=None,
             gate=None) -> torch.Tensor:
    """A packed batch of d.batch prompts (checked lengths; token arrays [sum][H][..]) through the
    layer, from `state` and into it; returns its outputs [sum][H][d_v]."""
    total, make = q.shape[0], _new_rows(lengths)
    plan = _plan(lengths, total, state.device)
    if conv is not None:
        q, k, v = conv._prefill(plan, torch.empty, (q, k, v))
    y = make((total, d.heads, d.d_v), device=state.device, dtype=torch.float32)
    scan_forward(d, total, plan, q, k, v, decay, beta, state, y, state_in=state)
    if norm is not None:
        y = norm(y, gate)
        if make is torch.zeros:  # the norm of a row of zeros need not be zero
            behind = torch.arange(total, device=state.device) >= plan[d.batch]
            y.masked_fill_(behind[:, None, None], 0.0)
    return y


class WindowedDecoder:
    """One layer's decode state on one device.

    state:  fp32 [N, H, d_k, d_v] (used in place: the decoder writes it once per window)
    basis:  fp32 [H, r, d_k] with orthonormal rows, or None for the exact-read path only
    read:   "sketch" (the SketchSSM read), "full" (the exact buffered read, no
            sketch kept) or "both" (both reads of the same tokens; for checks)
    fused:  append the current token inside the read kernel instead of a
            separate buffering launch
    ranks:  optional per-head sketch ranks (H values); then basis is fp32 [sum(ranks), d_k]
            and the sketch [N, sum(ranks), d_v]
    coefficients: "projection" (c = B q~) or "least_squares" (c minimising the error of the
            window-start read; then `sketch` holds orthonormal sketch rows and `read_map`
            [N, H, r, d_k] the per-unit map q~ -> c; uniform rank and fp32 sketch only)
    conv, norm: the layer's short convolution and output norm, or None. With a convolution q, k, v are the
            projections that go into it (rows of H d_k, H d_k and H d_v channels; they may be column ranges of
            one tensor); with a norm the outputs are normalised and gated by `gate`, in its in_dtype. The norm's groups
            divide the H d_v channels of a token as they like: heads, runs of heads, all of them.
    The sketch is kept in dims.sketch_dtype (fp32, or bf16 rounded to nearest).
    """

    def __init__(self, dims: Dims, state: torch.Tensor, basis: Optional[torch.Tensor] = None, *,
                 read: str = "sketch", fused: bool = True, ranks=None,
                 coefficients: str = "projection", conv: Optional[ShortConv] = None,
                 norm: Optional[GatedNorm] = None):
        if read not in ("sketch", "full", "both"):
            raise ValueError(read)
        if coefficients not in ("projection", "least_squares"):
            raise ValueError(coefficients)
        self.ls = coefficients == "least_squares"
        if self.ls and ranks is not None:
            raise ValueError("least-squares coefficients use a uniform rank")
        if read != "full" and basis is None:
            raise ValueError("a sketch read needs a basis")
        if norm is not None and read == "both":
            raise ValueError("two reads are compared before the norm")
        _around(dims, conv, norm)
        self.conv, self.norm = conv, norm
        self.d = dims
        self.read = read
        self.fused = fused
        dev = state.device
        N, H, dk, dv, W, r = dims.batch, dims.heads, dims.d_k, dims.d_v, dims.window, dims.rank
        tin = torch.bfloat16 if dims.in_dtype == IN_BF16 else torch.float32
        self.state = state
        self.basis = basis
        self.offsets = rank_offsets(ranks) if ranks is not None else None
        rows = (H, r) if ranks is None else (int(self.offsets[H]),)
        sk_dtype = torch.bfloat16 if dims.sketch_dtype == SKETCH_BF16 else torch.float32
        self.sketch = (torch.empty((N,) + rows + (dv,), device=dev, dtype=sk_dtype)
                       if read != "full" else None)
        self.read_map = (torch.empty((N, H, r, dk), device=dev, dtype=torch.float32)
                         if self.ls and read != "full" else None)
        self.k_buf = torch.zeros((N, H, W, dk), device=dev, dtype=tin)
        self.v_buf = torch.zeros((N, H, W, dv), device=dev, dtype=tin)
        dshape = (N, H, W, dk) if dims.rule == KDA else (N, H, W)
        self.decay_buf = torch.zeros(dshape, device=dev, dtype=torch.float32)
        self.beta_buf = (torch.zeros((N, H, W), device=dev, dtype=torch.float32)
                         if dims.rule != MAMBA2 else None)
        self._placed = (), []  # the buffers, and where they lie
        self.tau = 0  # tokens already in the window buffer

    # -- library calls, uniform or per-head ranks --------------------------------
    def _update(self, n_tokens: int) -> None:
        bufs = (self.k_buf, self.v_buf, self.decay_buf, self.beta_buf)
        if n_tokens == 0:
            bufs = (None, None, None, None)
        if self.read_map is not None:
            window_update_refresh_ls(self.d, self.state, self.sketch, self.read_map, self.basis,
                                     *bufs, n_tokens)
        elif self.offsets is not None and self.sketch is not None:
            window_update_refresh_ranked(self.d, self.offsets, self.state, self.sketch, self.basis,
                                         *bufs, n_tokens)
        else:
            window_update_refresh(self.d, self.state, self.sketch,
                                  self.basis if self.sketch is not None else None, *bufs, n_tokens)

    def _sketch_read(self, q, tau, y, tok) -> None:
        bufs = (self.k_buf, self.v_buf, self.decay_buf, self.beta_buf)
        if self.read_map is not None:
            sketch_decode_step_ls(self.d, self.sketch, self.read_map, q, *bufs, tau, y, **tok)
        elif self.offsets is not None:
            sketch_decode_step_ranked(self.d, self.offsets, self.sketch, self.basis, q, *bufs, tau,
                                      y, **tok)
        else:
            sketch_decode_step(self.d, self.sketch, self.basis, q, *bufs, tau, y, **tok)

    # -- window boundary ---------------------------------------------------------
    def refresh(self) -> None:
        """Store the sketch of the current state (refresh-only pass)."""
        if self.sketch is not None:
            self._update(0)

    def flush(self) -> None:
        """Write the buffered tokens into the state now (a partial window) and refresh."""
        self._update(self.tau)
        self.tau = 0

    # -- prompts -----------------------------------------------------------------
    def prefill(self, lengths, q, k, v, decay, beta=None, *, gate=None) -> torch.Tensor:
        """Take a packed batch of prompts (integer lengths [N], zero for a sequence with no new
        tokens; token arrays [sum of lengths][H][..]) into the state and refresh the sketch; returns
        the outputs [sum of lengths][H][d_v]. Tokens still in the window are written first. Lengths on
        the device are not read back: prompts are cut where the token arrays end, and outputs
        behind the last prompt are zero."""
        lengths = _checked_lengths(self.d, lengths, q)
        _prefill_check(self.d, q.shape[0], self.conv, self.norm, decay, beta, gate, self.state)
        with torch.cuda.device_of(self.state):  # the flush and the refresh on the scan's stream
            if self.tau:
                self.flush()
            y = _prefill(self.d, self.state, lengths, q, k, v, decay, beta, self.conv, self.norm, gate)
            self.refresh()
        return y

    # -- one decode step -----------------------------------------------------------
    def step(self, q, k, v, decay, beta=None, *, gate=None, y=None, y_full=None):
        """Read the output for the current token; returns y (or (y, y_full) for read="both"), or with a
        norm what the norm makes of it."""
        if _elsewhere(self):
            with torch.cuda.device_of(self.state):
                return self.step(q, k, v, decay, beta, gate=gate, y=y, y_full=y_full)
        d = self.d
        tau = self.tau + 1
        bufs = (self.k_buf, self.v_buf, self.decay_buf, self.beta_buf)
        if ((self.conv is not None or self.norm is not None)
                and (len(self._placed[0]) != 4 or not all(map(operator.is_, bufs, self._placed[0])))):
            self._placed = bufs, [_whole(t) for t in bufs if t is not None]
        _check_around(d, d.batch, self.conv, self.norm, decay, beta, gate, self.state, written=self._placed[1],
                      kept=(self.sketch, self.basis, self.read_map), ys=(y, y_full))
        if self.conv is not None:
            q, k, v = self.conv.step(q, k, v)
        N, H, dv = d.batch, d.heads, d.d_v
        if y is None and self.read != "full":
            y = torch.empty((N, H, dv), device=q.device, dtype=torch.float32)
        if y_full is None and self.read != "sketch":
            y_full = torch.empty((N, H, dv), device=q.device, dtype=torch.float32)
        tok = dict(k_t=k, v_t=v, decay_t=decay, beta_t=beta)
        if not self.fused:
            buffer_append(d, k, v, decay, beta, self.k_buf, self.v_buf, self.decay_buf,
                          self.beta_buf, tau - 1)
            tok = {}
        if self.read != "full":
            self._sketch_read(q, tau, y, tok)
            tok = {}  # the token is in the buffer now
        if self.read != "sketch":
            full_read_decode_step(d, self.state, q, *bufs, tau, y_full, **tok)
        self.tau = tau
        if tau == d.window:
            self._update(tau)
            self.tau = 0
        if self.read == "both":
            return y, y_full
        y = y if self.read == "sketch" else y_full
        return y if self.norm is None else self.norm(y, gate)


class RecurrentDecoder:
    """The per-token recurrent decode (the baseline SketchSSM is compared against):
    every step writes the token into the full state and reads y = S^T q from it.
    conv, norm: as in WindowedDecoder."""

    def __init__(self, dims: Dims, state: torch.Tensor, *, conv: Optional[ShortConv] = None,
                 norm: Optional[GatedNorm] = None):
        _around(dims, conv, norm)
        self.d, self.state, self.conv, self.norm = dims, state, conv, norm

    def step(self, q, k, v, decay, beta=None, *, gate=None, y=None):
        if _elsewhere(self):
            with torch.cuda.device_of(self.state):
                return self.step(q, k, v, decay, beta, gate=gate, y=y)
        d = self.d
        _check_around(d, d.batch, self.conv, self.norm, decay, beta, gate, self.state, ys=(y,))
        if self.conv is not None:
            q, k, v = self.conv.step(q, k, v)
        if y is None:
            y = torch.empty((d.batch, d.heads, d.d_v), device=q.device, dtype=torch.float32)
        recurrent_decode_step(d, self.state, q, k, v, decay, beta, y)
        return y if self.norm is None else self.norm(y, gate)

    def prefill(self, lengths, q, k, v, decay, beta=None, *, gate=None) -> torch.Tensor:
        """Take a packed batch of prompts into the state; returns their outputs (lengths and
        outputs as in WindowedDecoder.prefill)."""
        lengths = _checked_lengths(self.d, lengths, q)
        _prefill_check(self.d, q.shape[0], self.conv, self.norm, decay, beta, gate, self.state)
        with torch.cuda.device_of(self.state):
            return _prefill(self.d, self.state, lengths, q, k, v, decay, beta, self.conv, self.norm, gate)


class SelectiveDecoder:
    """One selective layer's recurrence for dims.batch sequences.

    state:  fp32 [batch, channels, d_state], used in place
    A:      fp32 [channels, d_state] (negative), D and dt_bias fp32 [channels] or None
    """

    def __init__(self, dims: SelectiveDims, state: torch.Tensor, A: torch.Tensor, *,
                 D: Optional[torch.Tensor] = None, dt_bias: Optional[torch.Tensor] = None):
        self.d, self.state, self.A = dims, state, A
        self.more = {"D": D, "dt_bias": dt_bias}

    def step(self, x, dt, B, C, z=None, *, out=None) -> torch.Tensor:
        """One token of every sequence: x, dt, z [batch][channels], B, C [batch][groups][d_state];
        returns out [batch][channels]."""
        d = self.d
        if out is None:
            out = torch.empty((d.batch, d.channels), device=x.device, dtype=_in_type(d.in_dtype))
        selective_step(d, x, dt, self.A, B, C, self.state, out, z=z, **self.more)
        return out

    def prefill(self, lengths, x, dt, B, C, z=None) -> torch.Tensor:
        """Take a packed batch of prompts (rows [sum of lengths][..]) into the state; returns their outputs
        (lengths and outputs as in WindowedDecoder.prefill)."""
        d, total = self.d, x.shape[0]
        lengths = _checked_lengths(d, lengths, x)
        with torch.cuda.device_of(self.state):
            plan = _plan(lengths, total, self.state.device)
            out = _new_rows(lengths)((total, d.channels), device=self.state.device, dtype=_in_type(d.in_dtype))
            selective_forward(d, total, plan, x, dt, self.A, B, C, self.state, out, z=z, state_in=self.state,
                              **self.more)
        return out
