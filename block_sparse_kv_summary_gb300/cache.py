"""Device buffers of a CompKV cache, allocated with PyTorch, driven through the C ABI.

PyTorch provides the device memory and the stream; each method checks its
tensors (device, dtype, shape, contiguity) and passes their addresses to the
library.  Nothing here computes any part of the decode step.
"""
from __future__ import annotations

import torch

from . import compkv as C

BLOCK = 16


_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _stream(device) -> int:
    return _raw_stream(device.index)


_TYPES = {torch.bfloat16: C.COMPKV_BF16, torch.float32: C.COMPKV_F32}


class CompKVCache:
    """A CompKV cache of `num_layers` layers x `batch` sequences on one GPU.

    capacity_tokens: an int (every sequence) or a list (ragged), multiples of 16.
    kv_memory: "device" (the K and V rows in GPU memory, the default) or "host"
        (in page-locked host memory, which the GPU reads over its chip-to-chip
        link; the summaries, the scratch and everything else stay in GPU memory).
    """

    def __init__(self, *, num_layers, batch, num_kv_heads, group_size, head_dim, r,
                 budget_tokens, capacity_tokens, device="cuda", variant=0, kv_memory="device"):
        self.device = torch.device(device)
        if self.device.type != "cuda":
            raise RuntimeError("CompKVCache lives in GPU memory; the library has no CPU path")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        caps = [capacity_tokens] * batch if isinstance(capacity_tokens, int) else list(capacity_tokens)
        self.cfg = C.make_config(num_layers, batch, num_kv_heads, group_size, head_dim, r,
                                 budget_tokens, capacity_tokens=caps, variant=variant)
        self.variant = variant
        self.num_layers, self.batch, self.Hkv, self.G = num_layers, batch, num_kv_heads, group_size
        self.d, self.r, self.K = head_dim, r, budget_tokens // BLOCK
        self.caps = caps
        self.max_cap_blocks = max(caps) // BLOCK
        rows = C.compkv_rows_per_layer(self.cfg)
        if rows <= 0:
            raise C.CompKVError(2, C.compkv_last_error())
        self.rows_per_layer = rows
        total = rows * num_layers
        dev = self.device
        if kv_memory not in ("device", "host"):
            raise ValueError(f"kv_memory must be 'device' or 'host', got {kv_memory!r}")
        self.kv_memory = kv_memory
        if kv_memory == "host":
            self.k = torch.zeros((total, BLOCK, head_dim), dtype=torch.bfloat16, pin_memory=True)
            self.v = torch.zeros((total, BLOCK, head_dim), dtype=torch.bfloat16, pin_memory=True)
        else:
            self.k = torch.zeros((total, BLOCK, head_dim), dtype=torch.bfloat16, device=dev)
            self.v = torch.zeros((total, BLOCK, head_dim), dtype=torch.bfloat16, device=dev)
        self.kbar = torch.zeros((total, head_dim), dtype=torch.float32, device=dev)
        self.vbar = torch.zeros((total, head_dim), dtype=torch.float32, device=dev)
        self.dbar = torch.zeros((total, r), dtype=torch.float32, device=dev)
        self.seq_len = torch.zeros((num_layers, batch), dtype=torch.int32, device=dev)
        nbytes = C.compkv_scratch_bytes(self.cfg)
        self.scratch = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        self.bufs = C.compkv_buffers(self.k.data_ptr(), self.v.data_ptr(), self.kbar.data_ptr(),
                                     self.vbar.data_ptr(), self.dbar.data_ptr(),
                                     self.seq_len.data_ptr(), self.scratch.data_ptr(), nbytes)
        self._index = self.device.index
        self._shared_ws = None
        # shapes of a call's outputs, and of the rows of the projection that it reads
        self._q_shape, self._kv_shape = (batch, num_kv_heads * group_size, head_dim), (batch, num_kv_heads, head_dim)
        self._width = (group_size + 2) * num_kv_heads * head_dim
        with torch.cuda.device(dev):
            self.ctx = C.compkv_init(self.cfg, self.bufs)

    # ------------------------------------------------------------------ layout
    def rows(self, layer, seq, head):
        """(first row, capacity in blocks) of a (layer, sequence, head)."""
        return C.compkv_row_offset(self.ctx, layer, seq, head)

    def token_view(self, layer, seq, head):
        """Views [capacity_tokens, d] of the K and V tokens of one (layer, sequence, head)."""
        r0, cap = self.rows(layer, seq, head)
        return (self.k[r0:r0 + cap].view(cap * BLOCK, self.d),
                self.v[r0:r0 + cap].view(cap * BLOCK, self.d))

    def summary_view(self, layer, seq, head):
        r0, cap = self.rows(layer, seq, head)
        return self.kbar[r0:r0 + cap], self.dbar[r0:r0 + cap], self.vbar[r0:r0 + cap]

    # ------------------------------------------------------------------ checks
    def _t(self, t, name, dtype, shape):
        if t.device != self.device or t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
            raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)} on {self.device}, "
                             f"got {t.dtype} {tuple(t.shape)} on {t.device}")
        return t.data_ptr()

    def _q(self, q):
        return self._t(q, "q", torch.float32, (self.batch, self.Hkv * self.G, self.d))

    def _kv(self, t, name):
        return self._t(t, name, torch.bfloat16, (self.batch, self.Hkv, self.d))

    def new_sel(self):
        return torch.empty((self.batch, self.Hkv, self.K), dtype=torch.int32, device=self.device)

    def new_out(self):
        return torch.empty((self.batch, self.Hkv * self.G, self.d), dtype=torch.float32, device=self.device)

    # ------------------------------------------------------------------ calls
    def prefill(self, layer, lens):
        C.compkv_prefill(self.ctx, layer, [int(x) for x in lens], _stream(self.device))

    def append(self, layer, k_new, v_new):
        C.compkv_append(self.ctx, layer, self._kv(k_new, "k_new"), self._kv(v_new, "v_new"),
                        _stream(self.device))

    def score_select(self, layer, q, sel=None, scores=None):
        sel = self.new_sel() if sel is None else sel
        sp = 0
        if scores is not None:
            sp = self._t(scores, "scores", torch.float32, (self.batch, self.Hkv, self.max_cap_blocks))
        C.compkv_score_select(self.ctx, layer, self._q(q),
                              self._t(sel, "sel", torch.int32, (self.batch, self.Hkv, self.K)),
                              sp, _stream(self.device))
        return sel

    def attend(self, layer, q, sel, out=None):
        out = self.new_out() if out is None else out
        C.compkv_attend(self.ctx, layer, self._q(q),
                        self._t(sel, "sel", torch.int32, (self.batch, self.Hkv, self.K)),
                        self._t(out, "out", torch.float32, (self.batch, self.Hkv * self.G, self.d)),
                        _stream(self.device))
        return out

    def decode(self, layer, q, k_new, v_new, out=None, sel=None):
        out = self.new_out() if out is None else out
        sp = 0 if sel is None else self._t(sel, "sel", torch.int32, (self.batch, self.Hkv, self.K))
        C.compkv_decode(self.ctx, layer, self._q(q), self._kv(k_new, "k_new"), self._kv(v_new, "v_new"),
                        self._t(out, "out", torch.float32, (self.batch, self.Hkv * self.G, self.d)),
                        sp, _stream(self.device))
        return out

    def prepared_decode(self):
        """A compkv_decode bound to this cache's context and the current stream:
        call it with (layer, q_ptr, k_ptr, v_ptr, out_ptr, sel_ptr) as plain
        device addresses; no per-call tensor checks."""
        return C.PreparedDecode(self.ctx, _stream(self.device))

    def decode_host(self, layer, q, k_new, v_new, out, sel=None):
        """compkv_decode_host on CPU tensors (q fp32 [B][Hq][d], k_new/v_new bf16
        [B][Hkv][d], out fp32 [B][Hq][d], sel int32 [B][Hkv][K] or None); returns
        when out is filled.  Page-locked tensors are read and written by the
        kernels directly; others are copied."""
        for t, name in ((q, "q"), (k_new, "k_new"), (v_new, "v_new"), (out, "out")):
            if t.device.type != "cpu" or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous CPU tensor")
        C.compkv_decode_host(self.ctx, layer, q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), out.data_ptr(),
                             0 if sel is None else sel.data_ptr(), _stream(self.device))
        return out

    # ------------------------------------------------------------------ around the decode step
    # (these calls take microseconds, so their checks are written out for speed)
    def _call(self, fn, *args):
        """A library call with the cache's device as the current one."""
        index = self._index
        if _current_device() == index:
            fn(self.ctx, *args, _raw_stream(index))
        else:
            with torch.cuda.device(index):
                fn(self.ctx, *args, _raw_stream(index))

    def _is(self, t, name, dtype, shape):
        """Address of a contiguous tensor of this type and shape."""
        if t.dtype is not dtype or t.shape != shape or t.device != self.device or not t.is_contiguous():
            self._t(t, name, dtype, shape)
        return t.data_ptr()

    def _rope_args(self, qkv, tokens, table, q_weight, k_weight, eps, positions, interleaved, q_dtype):
        width, dev, d = self._width, self.device, (self.d,)
        if q_dtype not in _TYPES:
            raise ValueError(f"q_dtype must be torch.float32 or torch.bfloat16, got {q_dtype}")
        if table.dim() != 2:
            raise ValueError(f"table must be [positions, rot_dim], got {tuple(table.shape)}")
        stride = qkv.stride()
        if (qkv.dtype not in _TYPES or qkv.shape != (tokens, width) or qkv.device != dev
                or stride[1] != 1 or (tokens > 1 and stride[0] < width)):
            raise ValueError(f"qkv: expected rows {(tokens, width)} of {' or '.join(map(str, _TYPES))} on {dev}, "
                             f"got {qkv.dtype} {tuple(qkv.shape)} with strides {stride} on {qkv.device}")
        positions_rows, rot = table.shape
        if table.dtype is not torch.float32 or table.device != dev or not table.is_contiguous():
            self._t(table, "table", torch.float32, table.shape)
        return C.compkv_rope_args(
            qkv.data_ptr(), _TYPES[qkv.dtype], stride[0] if tokens > 1 else width, table.data_ptr(), positions_rows, rot,
            1 if interleaved else 0, None if q_weight is None else self._is(q_weight, "q_weight", torch.float32, d),
            None if k_weight is None else self._is(k_weight, "k_weight", torch.float32, d), eps,
            None if positions is None else self._is(positions, "positions", torch.int32, (tokens,)), _TYPES[q_dtype])

    def rope(self, layer, qkv, table, *, q_weight=None, k_weight=None, eps=1e-6, positions=None, interleaved=False,
             q_dtype=torch.float32, q=None, k_new=None, v_new=None):
        """Norms and rotation of one token per sequence: (q, k_new, v_new) for decode.

        qkv: [B, (Hq + 2 Hkv) d] bf16 or fp32 (rows may stand apart); table: fp32 [positions, rot_dim], cos then
        sin of every position; q_weight, k_weight: fp32 [d] or None (no norm); positions: int32 [B] or None (the
        sequences' lengths).  See include/compkv.h."""
        a = self._rope_args(qkv, self.batch, table, q_weight, k_weight, eps, positions, interleaved, q_dtype)
        if q is None:
            q = torch.empty(self._q_shape, dtype=q_dtype, device=self.device)
        else:
            self._is(q, "q", q_dtype, self._q_shape)
        if k_new is None:
            k_new = torch.empty(self._kv_shape, dtype=torch.bfloat16, device=self.device)
        else:
            self._is(k_new, "k_new", torch.bfloat16, self._kv_shape)
        if v_new is None:
            v_new = torch.empty_like(k_new)
        else:
            self._is(v_new, "v_new", torch.bfloat16, self._kv_shape)
        self._call(C.compkv_rope, layer, a, q.data_ptr(), k_new.data_ptr(), v_new.data_ptr())
        return q, k_new, v_new

    def prefill_qkv(self, layer, qkv, counts, table, *, starts=None, q_weight=None, k_weight=None, eps=1e-6,
                    positions=None, interleaved=False, q_dtype=torch.float32, q=None):
        """Norms and rotation of many tokens, packed into the cache with their summaries; returns the queries.

        qkv: [tokens, (Hq + 2 Hkv) d], the counts[s] tokens of every sequence one after another; they go to the
        slots from starts[s] (0) on.  positions: int32 [tokens] or None (the slots)."""
        counts, starts = C.ints(counts), C.ints(starts)
        if len(counts) != self.batch or (starts is not None and len(starts) != self.batch):
            raise ValueError(f"counts and starts need {self.batch} entries")
        tokens = sum(counts)
        if min(counts) < 0:
            raise ValueError(f"counts must not be negative, got {counts.tolist()}")
        shape = (tokens, self.Hkv * self.G, self.d)
        a = self._rope_args(qkv, tokens, table, q_weight, k_weight, eps, positions, interleaved, q_dtype)
        if q is None:
            q = torch.empty(shape, dtype=q_dtype, device=self.device)
        else:
            self._is(q, "q", q_dtype, shape)
        if tokens:
            self._call(C.compkv_prefill_qkv, layer, a, starts, counts, q.data_ptr())
        return q

    def _pairs(self, src, dst, layers):
        src = C.ints(src)
        dst = src if dst is None else C.ints(dst)
        if len(src) != len(dst):
            raise ValueError(f"src and dst must have one entry per pair, got {len(src)} and {len(dst)}")
        layer0, n = (0, self.num_layers) if layers is None else (int(layers[0]), int(layers[1]) - int(layers[0]))
        return src, dst, layer0, n

    def fork(self, src, dst, lens=None, layers=None):
        """Copy the first lens[i] tokens (None or -1: all) of sequence src[i] to dst[i], summaries included, in
        the layers [layers[0], layers[1]) (None: every layer); src[i] == dst[i] cuts it in place."""
        src, dst, layer0, n = self._pairs(src, dst, layers)
        lens = C.ints(lens)
        if lens is not None and len(lens) != len(src):
            raise ValueError(f"lens must have one entry per pair, got {len(lens)} for {len(src)}")
        self._call(C.compkv_fork, layer0, n, src, dst, lens)

    def truncate(self, seqs, lens, layers=None):
        """Cut sequences to lens[i] tokens in place (0 frees them)."""
        self.fork(seqs, seqs, lens, layers)

    def compact(self, keep, src=None, dst=None, layers=None):
        """Keep only the listed blocks: keep int32 [layers, pairs, Hkv, M] ascending, padded with -1 (a selection's
        format); block keep[.., j] of sequence src[i] (None: every sequence) becomes block j of dst[i] (None: in
        place)."""
        src, dst, layer0, n = self._pairs(range(self.batch) if src is None else src, dst, layers)
        if keep.dim() != 4:
            raise ValueError(f"keep must be [layers, pairs, Hkv, blocks], got {tuple(keep.shape)}")
        kp = self._is(keep, "keep", torch.int32, (n, len(src), self.Hkv, keep.shape[3]))
        self._call(C.compkv_compact, layer0, n, src, dst, kp, keep.shape[3])

    def shared_workspace(self):
        """The workspace of attend_shared, allocated on first use and kept."""
        if self._shared_ws is None:
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError("attend_shared needs its workspace before a capture: call shared_workspace() first")
            self._shared_ws = torch.empty(C.compkv_attend_shared_bytes(self.cfg), dtype=torch.uint8, device=self.device)
        return self._shared_ws

    def attend_shared(self, layer, q, prefix_seq, prefix_len, out=None):
        """Exact attention over a prefix that sequence prefix_seq[s] holds for sequence s (its first
        prefix_len[prefix_seq[s]] tokens) and over the sequence's own tokens; -1: no prefix, -2: no part.
        q: [B, Hq, d] fp32 or bf16; out has its type.  With fp32, queries and softmax weights keep 24 bits; with bf16,
        the weights too are rounded to bf16, each by up to 2^-8 of itself, before they multiply the values (their sum
        is that of the rounded ones)."""
        prefix_seq, prefix_len = C.ints(prefix_seq), C.ints(prefix_len)
        if len(prefix_seq) != self.batch or len(prefix_len) != self.batch:
            raise ValueError(f"prefix_seq and prefix_len need {self.batch} entries")
        dtype, shape = q.dtype, self._q_shape
        if dtype not in _TYPES:
            raise ValueError(f"q must be torch.float32 or torch.bfloat16, got {dtype}")
        qp = self._is(q, "q", dtype, shape)
        if out is None:
            out = torch.empty_like(q)
        else:
            self._is(out, "out", dtype, shape)
        ws = self.shared_workspace()
        self._call(C.compkv_attend_shared, layer, qp, _TYPES[dtype], prefix_seq, prefix_len, out.data_ptr(),
                   ws.data_ptr(), ws.numel())
        return out

    def device_status(self) -> int:
        return C.compkv_device_status(self.ctx, _stream(self.device))

    def selftest_wait_timeout(self):
        C.compkv_selftest_wait_timeout(self.ctx, _stream(self.device))

    def launch_count(self) -> int:
        return C.compkv_launch_count(self.ctx)

    def profile(self, enable):
        C.compkv_profile_enable(self.ctx, enable)

    def profile_read(self, family):
        return C.compkv_profile_read(self.ctx, family)

    def close(self):
        if getattr(self, "ctx", None):
            C.compkv_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
