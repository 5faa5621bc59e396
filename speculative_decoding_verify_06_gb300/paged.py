"""Verify passes of several requests over a paged 4-bit cache, with the lengths kept on the GPU.

A step is what "100 tokens per second ..." ("How speculative decoding gets past a per-token wall")
describes for one sequence, for a batch of them ("Why a hiring company is writing this"): the tables
follow the tokens that the last acceptance kept (svd_paged_advance), every layer's queries and keys are
rotated and its keys and values appended (svd_paged_append), and the window's tokens attend to
their requests' caches (svd_paged_attention).  Nothing of a step waits for the host: acceptance
counts, lengths, page ids and free pages stay in device memory, at the same addresses in every step, so a step can
be recorded and replayed.

    python -m speculative_decoding_verify_06_gb300.paged [requests] [window] [steps]

runs a two-layer stand-in for a model on synthetic weights, accepting drafts and growing the caches.
"""
from __future__ import annotations

import contextlib

import torch

from . import svd


class PagedBatch:
    """The caches of `requests` requests in `layers` pools of n_pages pages, one table for all layers.

    A request has up to max_window tokens in a step (lowered where windows stay shorter: the attention then
    takes smaller tiles), all requests together max_tokens.

    begin() opens a step, layer() runs one layer's append and attention.  Between two begin() calls
    the device tensors q_start, kv_len, slots, positions and status describe the step's tokens; held and
    window are the state that the next begin() goes on from.  stream: a torch stream or its address, None for
    the current one; a tensor handed to a call stays alive until that stream has used it."""

    def __init__(self, requests: int, layers: int, n_pages: int, page_size: int = 64, max_len: int = 32768,
                 max_window: int = 8, n_q_heads: int = 40, n_kv_heads: int = 8, rope: svd.Rope | None = None,
                 out_dtype: int = svd.SVD_BF16, max_tokens: int | None = None, device="cuda"):
        dev = torch.device(device)
        self.device, self.R, self.page, self.n_pages = dev, requests, page_size, n_pages
        self.Hq, self.Hkv, self.rope, self.out_dtype = n_q_heads, n_kv_heads, rope, out_dtype
        self.width = -(-max_len // page_size)
        self.max_window = self._step_window = max_window
        self.max_tokens = max_tokens or requests * max_window
        nbytes = svd.svd_paged_cache_bytes(n_kv_heads, page_size, n_pages)
        if nbytes == 0:
            raise ValueError("no such pool: see svd_paged_cache_bytes")
        self.pools = [torch.zeros(nbytes, dtype=torch.uint8, device=dev) for _ in range(layers)]
        i32 = dict(dtype=torch.int32, device=dev)
        # The state lies in one piece, so that the copy that a step writes takes one transfer to become the
        # copy that the next one reads; both stay where they are, so that a recorded step can be replayed.
        sizes = [requests * self.width, n_pages, 1, requests, requests]
        self._state = [torch.zeros(sum(sizes), **i32) for _ in range(2)]
        table, self.free, self.n_free, self.held, self._window = zip(*(c.split(sizes) for c in self._state))
        self.table = [t.view(requests, self.width) for t in table]
        self.now = 0  # the copy that holds the state between steps
        self.table[0].fill_(-1)
        self.free[0].copy_(torch.arange(n_pages - 1, -1, -1, **i32))  # page 0 on top
        self.n_free[0].fill_(n_pages)
        self.q_start = torch.zeros(requests + 1, **i32)
        self.slots = torch.full((self.max_tokens,), -1, dtype=torch.int64, device=dev)
        self.positions = torch.full((self.max_tokens,), -1, **i32)
        self.status = torch.zeros(requests, **i32)
        self.kv_len = torch.zeros(requests, **i32)
        self.ws = torch.zeros(svd.svd_paged_attention_workspace_bytes(n_q_heads, n_kv_heads, requests, max_window),
                              dtype=torch.uint8, device=dev)
        self.q = torch.empty((self.max_tokens, n_q_heads, 128), dtype=torch.bfloat16, device=dev)
        self.bad = torch.zeros(self.max_tokens, **i32)  # SVD_ST_* bits of the tokens appended since it was zeroed
        self.scale = 128 ** -0.5

    @property
    def window(self):
        """Tokens of the step whose count of kept ones the next begin() takes; -d once d positions are
        known to go."""
        return self._window[self.now]

    @property
    def attention_status(self):
        """int32 [1], 0 while all is well; bit 0: a bounded wait of an attention kernel gave up, outputs since then
        are undefined; bit 1: a finite query was above 65504 in magnitude, its row is NaN.  Stays until zeroed."""
        return self.ws[:4].view(torch.int32)

    def begin(self, n_new, emitted=None, stream=None):
        """Opens a step of n_new [R] new tokens for each request, after `emitted` [R] of the last
        step's tokens were kept (None: all of them; a request that had no tokens has no count).  Requests
        that cannot be served have a status and no tokens; they keep what they hold, and the count of their
        last window holds as given, unless it was out of order."""
        self._counts("n_new", n_new)
        if emitted is not None:
            self._counts("emitted", emitted)
        a, b = self.now, 1 - self.now
        self._step_window = self.max_window
        svd.svd_paged_advance(self.held[a], self._window[a], emitted, n_new, self.R, self.max_window, self.page, self.table[a],
                              self.width, self.free[a], self.n_free[a], self.n_pages, self.held[b], self._window[b], self.table[b],
                              self.free[b], self.n_free[b], self.kv_len, self.q_start, self.slots, self.positions,
                              self.max_tokens, self.status, stream=stream)
        with self._on(stream):
            self._state[a].copy_(self._state[b])

    def end(self, who, stream=None):
        """Requests (bool [R]) that are over: the next begin() gives all their pages back, and counts what it adds
        for them from position 0.  Comes after the last layer() of a step, in place of their kept counts."""
        self._here("who", who, torch.bool)
        if who.shape != (self.R,):
            raise ValueError(f"who: [{self.R}], got {tuple(who.shape)}")
        with self._on(stream):
            torch.where(who, -self.held[self.now], self.window, out=self.window)

    def _on(self, stream):
        if stream is None:
            return contextlib.nullcontext()
        if isinstance(stream, int):  # (an ExternalStream of 0 would be a new stream)
            dev = self.q_start.device
            stream = torch.cuda.ExternalStream(stream, device=dev) if stream else torch.cuda.default_stream(dev)
        return torch.cuda.stream(stream)

    def _here(self, name: str, t, *dtypes):
        """The library takes addresses: a tensor of another type or place would be read as it lies."""
        if t.dtype not in dtypes or t.device != self.q_start.device:
            raise ValueError(f"{name}: {' or '.join(str(d) for d in dtypes)} on {self.q_start.device}, got {t.dtype} on {t.device}")

    def _counts(self, name: str, t):
        self._here(name, t, torch.int32)
        if t.shape != (self.R,) or not t.is_contiguous():
            raise ValueError(f"{name}: [{self.R}] in one piece, got {tuple(t.shape)}")

    def _positions(self, positions, T: int):
        """The positions of layer() and the distance of their axes (0: one row for all of them)."""
        if positions is None:
            return self.positions, 0
        axes = 1 if self.rope is None else self.rope.n_axes
        self._here("positions", positions, torch.int32)
        if positions.dim() not in (1, 2) or positions.shape[-1] < T:
            raise ValueError(f"positions: [{axes}][{T}] or [{T}], got {tuple(positions.shape)}")
        if positions.dim() == 1:
            row, ld = positions, 0
        else:
            if positions.shape[0] < axes:
                raise ValueError(f"positions: {positions.shape[0]} axes, the rotary positions have {axes}")
            row, ld = positions[0], positions.stride(0) if axes > 1 else 0
        if row.shape[0] > 1 and row.stride(0) != 1:
            raise ValueError("positions: an axis lies in one piece")
        return positions, ld

    def layer(self, l: int, qkv, out, n_tokens: int | None = None, positions=None, stream=None):
        """Layer l's step: rotates and stores qkv [n_tokens][(Hq + 2 Hkv) * 128] (fp32, as
        svd_verify_linear writes it, or bf16) and writes its attention to out [n_tokens][Hq][128].
        positions, int32 [axes][n_tokens] (images: time, height, width) or [n_tokens] for all axes alike,
        replaces the requests' own positions, which are the same on every axis; the request of every token, for
        offsets of its own, is torch.searchsorted(q_start, arange, right=True) - 1.  n_tokens: the rows of qkv
        that count (None: all of them, up to max_tokens); it covers the step's tokens, q_start's last entry."""
        T = min(qkv.shape[0], self.max_tokens) if n_tokens is None else int(n_tokens)
        width = (self.Hq + 2 * self.Hkv) * 128
        if not 0 <= T <= self.max_tokens:
            raise ValueError(f"{T} tokens, the batch was made for {self.max_tokens}")
        self._here("qkv", qkv, torch.float32, torch.bfloat16)
        self._here("out", out, torch.float32 if self.out_dtype == svd.SVD_F32 else torch.bfloat16)
        if qkv.dim() != 2 or qkv.shape[0] < T or qkv.shape[1] < width or qkv.stride(1) != 1:
            raise ValueError(f"qkv: {T} rows of {width}, got {tuple(qkv.shape)} with strides {qkv.stride()}")
        if out.numel() < T * self.Hq * 128 or not out.is_contiguous():
            raise ValueError(f"out: [{T}][{self.Hq}][128] in one piece, got {tuple(out.shape)}")
        pos, pos_ld = self._positions(positions, T)
        if T == 0:
            return out
        pool = self.pools[l]
        svd.svd_paged_append(qkv, qkv.stride(0) if T > 1 else width, T, self.Hq, self.Hkv, self.slots, pool, self.page, self.n_pages, self.q,
                             rope=self.rope, positions=pos, positions_ld=pos_ld,
                             dtype=svd.SVD_F32 if qkv.dtype == torch.float32 else svd.SVD_BF16, status=self.bad,
                             stream=stream)
        svd.svd_paged_attention(self.q, T, self.kv_len, self.q_start, self.R, self._step_window, self.table[self.now], self.width,
                                pool, self.page, self.n_pages, self.Hq, self.Hkv, self.scale, out, self.out_dtype, self.ws,
                                stream=stream)
        return out


def demo(requests: int = 8, window: int = 4, steps: int = 6, prompt: int = 200, layers: int = 2, seed: int = 0):
    """Batched verify steps of a stand-in model: per layer q|k|v and o products of 4-bit weights
    (svd_verify_linear over all requests' window columns) around the paged attention; acceptance counts
    are drawn instead of sampled.  Returns the PagedBatch and the kept lengths, step by step."""
    from . import stack, synth
    dev = torch.device("cuda")
    C = requests * window
    hidden, kv = synth.HIDDEN, synth.N_KV_HEADS * 128
    rope = svd.Rope([10000.0 ** (-i / 64) for i in range(64)])
    b = PagedBatch(requests, layers, n_pages=requests * (prompt + (steps + 1) * window) // 64 + 2 * requests, max_len=4096,
                   max_window=max(window, prompt), rope=rope, max_tokens=max(C, requests * prompt))
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    # the prompts: their keys and values arrive in one step of `prompt` tokens a request
    b.begin(torch.full((requests,), prompt, dtype=torch.int32, device=dev))
    qkv = torch.randn((requests * prompt, hidden + 2 * kv), generator=g, device=dev)
    o = torch.empty((b.max_tokens, b.Hq, 128), dtype=torch.bfloat16, device=dev)
    for l in range(layers):
        b.layer(l, qkv, o, n_tokens=requests * prompt)
    b.max_window = window
    lin = [(stack.Linear(hidden, hidden + 2 * kv, C, seed + 10 * l, dev), stack.Linear(hidden, hidden, C, seed + 10 * l + 1, dev))
           for l in range(layers)]
    ws = torch.zeros(max(svd.svd_verify_linear_workspace_bytes(x.in_f, x.out_f, C) for p in lin for x in p), dtype=torch.uint8,
                     device=dev)
    n_new = torch.full((requests,), window, dtype=torch.int32, device=dev)
    lengths, emitted = [b.kv_len.tolist()], None
    for _ in range(steps):
        b.begin(n_new, emitted)
        x = synth.activations_torch(C, hidden, seed, dev)
        for l, (qkv_lin, o_lin) in enumerate(lin):
            svd.svd_verify_linear(qkv_lin.W, x, C, qkv_lin.Y, ws)
            b.layer(l, qkv_lin.Y, o, n_tokens=C)
            svd.svd_verify_linear(o_lin.W, o, C, o_lin.Y, ws)  # the attention's bf16 is the product's input as it is
            x = (o_lin.Y / o_lin.Y.square().mean(-1, keepdim=True).sqrt()).to(torch.bfloat16)
        emitted = torch.randint(1, window + 1, (requests,), generator=g, device=dev).to(torch.int32)
        lengths.append((b.kv_len - window + emitted).tolist())
    return b, lengths


if __name__ == "__main__":
    import sys
    batch, kept = demo(*[int(a) for a in sys.argv[1:4]])
    for n, k in enumerate(kept):
        print(f"step {n}: kept positions {k}")
    print(f"{int(batch.n_free[batch.now])} of {batch.n_pages} pages free, status {batch.status.tolist()}")
