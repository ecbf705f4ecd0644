"""Torch-facing calls of the verify step: same names as the C ABI.

Each function only collects data pointers of CUDA tensors and the current
torch stream and calls libspecverify.so; the tensors must stay alive until the
stream has run the call (the argument structs keep references to them).
"""
import ctypes

import torch

from ._binding import (AdjustArgs, AttnArgs, COUNT_PROMPT, COUNT_RESET, CountArgs, DraftArgs,
                       ROPE_BANDED, ROPE_HALF, ROPE_INTERLEAVED, ROPE_LINEAR, ROPE_NTK,
                       ROPE_PLAIN, ROPE_YARN, RopeArgs, RopeScaling, SampleArgs, SV_BF16, SV_E4M3,
                       SV_F32, _check, lib)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _dt(t):
    if t.dtype == torch.bfloat16:
        return SV_BF16
    if t.dtype == torch.float32:
        return SV_F32
    if t.dtype == torch.uint8:          # E4M3 codes (an 8-bit KV cache)
        return SV_E4M3
    raise ValueError(f"unsupported dtype {t.dtype} (bfloat16, float32 or uint8 E4M3 codes)")


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def attn_args(q, k_new, v_new, k_cache, v_cache, cu_q, kv_start, kv_len, out, *, max_q_rows,
              kv_rows_bound, scale=0.0, dev_status=None, group=None, prefix_start=None,
              prefix_len=None, prefix_rows_bound=0, k_scale=0.0, v_scale=0.0):
    """sv_attn_args for q [R, Hq, D], k_new / v_new [R, Hkv, D], caches
    [P, Hkv, D], cu_q [B+1] int32, kv_start [B] int64, kv_len [B] int32,
    out [R, Hq, D]; max_q_rows / kv_rows_bound are host bounds.  Shared
    prefixes: group [B] int32 (non-decreasing), prefix_start [G] int64,
    prefix_len [G] int32 and the host bound prefix_rows_bound.  uint8 K/V
    tensors are E4M3 codes read as code * k_scale / code * v_scale."""
    a = AttnArgs()
    R, Hq, D = q.shape
    a.batch = cu_q.shape[0] - 1
    a.num_q_heads, a.num_kv_heads, a.head_dim = Hq, k_new.shape[1], D
    a.dtype = _dt(q)
    a.max_q_rows = int(max_q_rows)
    a.num_rows = R
    a.kv_rows_bound = int(kv_rows_bound)
    a.pool_rows = k_cache.shape[0]
    a.scale = float(scale)
    a.num_groups = 0 if group is None else prefix_len.shape[0]
    a.prefix_rows_bound = int(prefix_rows_bound)
    a.cu_q, a.q, a.k_new, a.v_new = _ptr(cu_q), _ptr(q), _ptr(k_new), _ptr(v_new)
    a.k_cache, a.v_cache = _ptr(k_cache), _ptr(v_cache)
    a.kv_start, a.kv_len, a.out = _ptr(kv_start), _ptr(kv_len), _ptr(out)
    a.dev_status = _ptr(dev_status)
    a.kv_dtype = SV_E4M3 if k_cache.dtype == torch.uint8 else 0
    a.k_scale, a.v_scale = float(k_scale), float(v_scale)
    a.group, a.prefix_start, a.prefix_len = _ptr(group), _ptr(prefix_start), _ptr(prefix_len)
    a._keep = (q, k_new, v_new, k_cache, v_cache, cu_q, kv_start, kv_len, out, dev_status,
               group, prefix_start, prefix_len)
    return a


def sample_args(target_logits, draft_logits, draft_tokens, cu_q, kv_len, num_accepted,
                out_tokens, *, max_q_rows, temperature, top_p, seed, seq_ids=None,
                dev_status=None, top_k=0, temperatures=None, top_ps=None, top_ks=None):
    """sv_sample_args for target_logits [R, V], draft_logits [R-B, V],
    draft_tokens [R-B] int32, cu_q [B+1], kv_len [B], outputs num_accepted [B]
    and out_tokens [R] (int32), seq_ids [B] int64 or None.  temperature 0 is
    greedy; top_k 0 disables top-k; temperatures / top_ps ([B] float32) and
    top_ks ([B] int32) override the scalars per sequence."""
    s = SampleArgs()
    R, V = target_logits.shape
    s.batch = cu_q.shape[0] - 1
    s.vocab = V
    s.dtype = _dt(target_logits)
    s.max_q_rows = int(max_q_rows)
    s.num_rows = R
    s.temperature = float(temperature)
    s.top_p = float(top_p)
    s.seed = int(seed) & 0xFFFFFFFFFFFFFFFF
    s.cu_q, s.target_logits = _ptr(cu_q), _ptr(target_logits)
    s.draft_logits = _ptr(draft_logits) if draft_logits.numel() else None
    s.draft_tokens = _ptr(draft_tokens) if draft_tokens.numel() else None
    s.kv_len, s.seq_ids = _ptr(kv_len), _ptr(seq_ids)
    s.num_accepted, s.out_tokens = _ptr(num_accepted), _ptr(out_tokens)
    s.dev_status = _ptr(dev_status)
    s.top_k = int(top_k)
    s.temperatures, s.top_ps, s.top_ks = _ptr(temperatures), _ptr(top_ps), _ptr(top_ks)
    s._keep = (target_logits, draft_logits, draft_tokens, cu_q, kv_len, seq_ids, num_accepted,
               out_tokens, dev_status, temperatures, top_ps, top_ks)
    return s


def draft_args(draft_logits, kv_len, draft_tokens, *, temperature, top_p, seed, seq_ids=None,
               dev_status=None, top_k=0, temperatures=None, top_ps=None, top_ks=None):
    """sv_draft_args for draft_logits [B, V] (one row per sequence), kv_len [B]
    (cache lengths before this position's append: row i's token sits at index
    kv_len[i] + 1), output draft_tokens [B] int32; parameters as in
    sample_args."""
    d = DraftArgs()
    B, V = draft_logits.shape
    d.batch, d.vocab, d.dtype = B, V, _dt(draft_logits)
    d.top_k = int(top_k)
    d.temperature, d.top_p = float(temperature), float(top_p)
    d.seed = int(seed) & 0xFFFFFFFFFFFFFFFF
    d.draft_logits, d.kv_len, d.seq_ids = _ptr(draft_logits), _ptr(kv_len), _ptr(seq_ids)
    d.temperatures, d.top_ps, d.top_ks = _ptr(temperatures), _ptr(top_ps), _ptr(top_ks)
    d.draft_tokens, d.dev_status = _ptr(draft_tokens), _ptr(dev_status)
    d._keep = (draft_logits, kv_len, seq_ids, temperatures, top_ps, top_ks, draft_tokens,
               dev_status)
    return d


def spec_draft_step(attn, draft, kv_cap, new_kv_len, ws, stream=None):
    """One draft position: single-row attention, append of the position's row
    and the draft-token draw, the last two beside the attention."""
    _check(lib.spec_draft_step(ctypes.byref(attn), ctypes.byref(draft), _ptr(kv_cap),
                               _ptr(new_kv_len), ctypes.c_void_p(ws.ptr), ws.nbytes,
                               _stream(stream)))


def draft_step_workspace_bytes(attn, draft):
    n = lib.sv_draft_step_workspace_bytes(ctypes.byref(attn), ctypes.byref(draft))
    if n == 0:
        _check(1)
    return n


def draft_workspace_bytes(draft):
    n = lib.sv_draft_workspace_bytes(ctypes.byref(draft))
    if n == 0:
        _check(1)
    return n


def workspace_bytes(attn=None, sample=None):
    n = lib.sv_workspace_bytes(ctypes.byref(attn) if attn is not None else None,
                               ctypes.byref(sample) if sample is not None else None)
    if n == 0:
        _check(1)
    return n


class Workspace:
    """A device workspace for the verify calls, zeroed once on creation."""

    def __init__(self, nbytes, device=None, stream=None):
        self.nbytes = int(nbytes)
        self.buf = torch.empty(self.nbytes + 256, dtype=torch.uint8, device=device or "cuda")
        base = self.buf.data_ptr()
        self.ptr = (base + 255) // 256 * 256
        _check(lib.sv_workspace_init(ctypes.c_void_p(self.ptr), self.nbytes, _stream(stream)))

    def zero(self, stream=None):
        """Zero the workspace again (after a call that reported SV_DEV_TIMEOUT)."""
        _check(lib.sv_workspace_init(ctypes.c_void_p(self.ptr), self.nbytes, _stream(stream)))

    @classmethod
    def for_args(cls, attn=None, sample=None, device=None, stream=None):
        return cls(workspace_bytes(attn, sample), device, stream)


def spec_verify_attn(attn, ws, stream=None):
    _check(lib.spec_verify_attn(ctypes.byref(attn), ctypes.c_void_p(ws.ptr), ws.nbytes,
                                _stream(stream)))


def spec_verify_attn_static(attn, stream=None):
    """spec_verify_attn with the library's static device scratch instead of a
    workspace, for callers that may not allocate device memory; nothing is
    allocated (the first call on a device sets the scratch up)."""
    _check(lib.spec_verify_attn_static(ctypes.byref(attn), _stream(stream)))


def sv_static_scratch_reset(stream=None):
    """Zero the static scratch's merge counters on `stream` (after a static call
    reported SV_DEV_TIMEOUT); allocates nothing."""
    _check(lib.sv_static_scratch_reset(_stream(stream)))


def sv_set_wait_limit(polls):
    """Bound on the polls of one attention pipeline wait (0: the built-in
    bound); a small bound makes waits run out on purpose (SV_DEV_TIMEOUT)."""
    _check(lib.sv_set_wait_limit(int(polls)))


def spec_reject_sample(sample, ws, stream=None):
    _check(lib.spec_reject_sample(ctypes.byref(sample), ctypes.c_void_p(ws.ptr), ws.nbytes,
                                  _stream(stream)))


def spec_draft_sample(draft, ws, stream=None):
    _check(lib.spec_draft_sample(ctypes.byref(draft), ctypes.c_void_p(ws.ptr), ws.nbytes,
                                 _stream(stream)))


def kv_append_ragged(cu_q, k_new, v_new, k_cache, v_cache, kv_start, kv_len, kv_cap,
                     num_accepted, new_kv_len, *, max_q_rows, dev_status=None, stream=None):
    B = cu_q.shape[0] - 1
    R, Hkv, D = k_new.shape
    _check(lib.kv_append_ragged(B, Hkv, D, _dt(k_new), int(max_q_rows), R, _ptr(cu_q),
                                _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                                k_cache.shape[0], _ptr(kv_start), _ptr(kv_len), _ptr(kv_cap),
                                _ptr(num_accepted), _ptr(new_kv_len), _ptr(dev_status),
                                _stream(stream)))


def spec_verify_step(attn, sample, kv_cap, new_kv_len, ws, stream=None):
    _check(lib.spec_verify_step(ctypes.byref(attn), ctypes.byref(sample), _ptr(kv_cap),
                                _ptr(new_kv_len), ctypes.c_void_p(ws.ptr), ws.nbytes,
                                _stream(stream)))


# ------------------------------------------------- operators around the step
_WORDS = (torch.int32, torch.uint32)        # 32-bit words of bits


class _Args:
    """Collects the tensors of one argument struct: every one on the same CUDA
    device, of the wanted dtype, with at least the wanted number of elements."""

    def __init__(self):
        self.device, self.keep = None, []

    def add(self, t, name, dtypes, shape=None, at_least=0, rows=False):
        if t is None:
            return None
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{name} must be a tensor on a CUDA device")
        if self.device is None:
            self.device = t.device
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, the other tensors on {self.device}")
        if t.dtype not in (dtypes if isinstance(dtypes, tuple) else (dtypes,)):
            raise ValueError(f"{name}: unsupported dtype {t.dtype}")
        if shape is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
        if t.numel() < at_least:
            raise ValueError(f"{name}: {t.numel()} elements, at least {at_least} needed")
        if not rows and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        self.keep.append(t)
        return t.data_ptr()


def _rows_stride(t, name):
    """Elements between the rows of [R, H, D], whose rows must be contiguous."""
    R, H, D = t.shape
    if (D > 1 and t.stride(2) != 1) or (H > 1 and t.stride(1) != D):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    if R <= 1:
        return H * D
    if t.stride(0) < H * D:
        raise ValueError(f"{name}: rows overlap")
    return t.stride(0)


def _launch(fn, args, stream):
    """Calls fn on `stream` or the current one; the tensors' device has to be the current one.
    (The raw stream: a torch.cuda.Stream object costs more than the launch.)"""
    device = args._device
    if torch._C._cuda_getDevice() != device:
        raise ValueError(f"tensors are on cuda:{device}, not on the current device")
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(device)
    elif stream.device_index != device:
        raise ValueError(f"tensors are on cuda:{device}, the stream on cuda:{stream.device_index}")
    else:
        raw = stream.cuda_stream
    st = fn(ctypes.byref(args), raw)
    if st:
        _check(st)


def _finish(a, c):
    """Keeps the tensors of an argument struct alive with it."""
    a._keep, a._device = c.keep, c.device.index
    return a


def rope_turns(rot_dim, *, base=10000.0, scaling="plain", factor=1.0, trained_len=1,
               beta_fast=0.0, beta_slow=0.0, low_freq=0.0, high_freq=0.0, device=None):
    """(turns, mscale): the table spec_rope_rows takes ([rot_dim / 2] int64
    holding 64-bit fractions of a turn per token) and the factor on cos and
    sin.  scaling: "plain", "linear", "ntk", "yarn" or "banded", for contexts
    `factor` times the trained one (spec_ops.h has the formulas)."""
    kinds = {"plain": ROPE_PLAIN, "linear": ROPE_LINEAR, "ntk": ROPE_NTK, "yarn": ROPE_YARN,
             "banded": ROPE_BANDED}
    if scaling not in kinds:
        raise ValueError(f"scaling {scaling!r} (one of {', '.join(kinds)})")
    sc = RopeScaling(kinds[scaling], int(trained_len), float(base), float(factor),
                     float(beta_fast), float(beta_slow), float(low_freq), float(high_freq))
    host = (ctypes.c_uint64 * max(1, int(rot_dim) // 2))()
    m = ctypes.c_float()
    _check(lib.sv_rope_turns(ctypes.byref(sc), int(rot_dim), host, ctypes.byref(m)))
    turns = torch.frombuffer(bytearray(host), dtype=torch.int64)
    return turns.to(device or "cuda"), m.value


def rope_args(q, k, v, q_out, k_out, v_out, turns, *, cu_q=None, kv_len=None, positions=None,
              max_q_rows=0, layout="half", mscale=1.0, k_scale=0.0, v_scale=0.0, dev_status=None):
    """sv_rope_args for q [R, Hq, D], k / v [R, Hkv, D] (rows may lie apart, as
    in a fused projection; any of the three may be None) and their contiguous
    outputs; turns [rot_dim / 2] int64 from rope_turns.  Positions: row j of
    sequence i at kv_len[i] + j with cu_q [B+1] and kv_len [B] (int32) and the
    host bound max_q_rows on a sequence's rows, or `positions` [R] int64.
    layout "half" (pairs rot_dim / 2 apart) or "interleaved" (neighbours).
    uint8 k_out / v_out take E4M3 codes of k / k_scale and v / v_scale."""
    a, c = RopeArgs(), _Args()
    first = next((t for t in (q, k, v) if t is not None), None)
    if first is None:
        raise ValueError("q, k and v are all None")
    if any(t is not None and t.dim() != 3 for t in (q, k, v)):
        raise ValueError("q, k and v must be [rows, heads, head_dim]")
    R, _, D = first.shape
    floats = (torch.bfloat16, torch.float32)
    if first.dtype not in floats:
        raise ValueError(f"unsupported dtype {first.dtype} (bfloat16 or float32)")
    for name, t, out in (("q", q, q_out), ("k", k, k_out), ("v", v, v_out)):
        if t is None:
            continue
        if out is None:
            raise ValueError(f"{name}_out is None")
        if t.shape[0] != R or t.shape[2] != D:
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected ({R}, heads, {D})")
        setattr(a, name, c.add(t, name, first.dtype, rows=True))
        setattr(a, name + "_out", c.add(out, name + "_out", (first.dtype,) if name == "q" else
                                        (first.dtype, torch.uint8), shape=t.shape))
        setattr(a, name + "_stride", _rows_stride(t, name))
    outs = {t.dtype for t, x in ((k_out, k), (v_out, v)) if x is not None}
    if len(outs) > 1 or (k is not None and v is not None and k.shape != v.shape):
        raise ValueError("k and v (and their outputs) must have one shape and dtype")
    if layout not in ("half", "interleaved"):
        raise ValueError(f"layout {layout!r} (half or interleaved)")
    a.num_q_heads = q.shape[1] if q is not None else 0
    a.num_kv_heads = next((t.shape[1] for t in (k, v) if t is not None), 0)
    a.head_dim, a.rot_dim, a.num_rows = D, 2 * turns.shape[0], R
    a.layout = ROPE_HALF if layout == "half" else ROPE_INTERLEAVED
    a.dtype = _dt(first)
    a.kv_dtype = SV_E4M3 if torch.uint8 in outs else 0
    a.mscale, a.k_scale, a.v_scale = float(mscale), float(k_scale), float(v_scale)
    a.turns = c.add(turns, "turns", torch.int64)
    if positions is not None:
        if cu_q is not None or kv_len is not None:
            raise ValueError("positions stand instead of cu_q and kv_len")
        a.positions = c.add(positions, "positions", torch.int64, shape=(R,))
        a.max_q_rows = 1        # (no rows: an empty tensor's null says by sequences)
    else:
        if cu_q is None or kv_len is None:
            raise ValueError("cu_q and kv_len, or positions, are needed")
        a.batch, a.max_q_rows = cu_q.shape[0] - 1, int(max_q_rows)
        a.cu_q = c.add(cu_q, "cu_q", torch.int32)
        a.kv_len = c.add(kv_len, "kv_len", torch.int32, shape=(a.batch,))
    a.dev_status = c.add(dev_status, "dev_status", _WORDS, at_least=1)
    return _finish(a, c)


def spec_rope_rows(rope, stream=None):
    """Rotates q and k (and turns k and v into cache codes) of every row."""
    _launch(lib.spec_rope_rows, rope, stream)


class TokenCounts:
    """A table of the tokens that `num_slots` requests have had, empty at first:
    `counts` [num_slots, vocab] int32 and `seen` [num_slots, ceil(vocab / 32)]
    int32, changed by spec_count_tokens and read by spec_adjust_logits."""

    def __init__(self, num_slots, vocab, device=None):
        device = device or "cuda"
        self.counts = torch.zeros(num_slots, vocab, dtype=torch.int32, device=device)
        self.seen = torch.zeros(num_slots, (vocab + 31) // 32, dtype=torch.int32, device=device)


def count_args(counts, seen, tokens, start, *, num_accepted=None, slots=None, prompt=False,
               reset=False, dev_status=None):
    """sv_count_args for the table counts [S, V] / seen [S, ceil(V / 32)],
    tokens [T] int32 and start [B+1] int32 (a step's out_tokens and cu_q, with
    its num_accepted: the first num_accepted + 1 of a sequence count).  prompt
    marks the tokens as a prompt's instead of counting them; reset clears the
    batch's slots first.  slots [B] int32: rows of the table (None: 0..B-1)."""
    a, c = CountArgs(), _Args()
    S, V = counts.shape
    B = start.shape[0] - 1
    a.batch, a.vocab, a.num_slots = B, V, S
    a.flags = (COUNT_PROMPT if prompt else 0) | (COUNT_RESET if reset else 0)
    a.num_tokens = tokens.numel()
    a.counts = c.add(counts, "counts", torch.int32)
    a.seen = c.add(seen, "seen", _WORDS, shape=(S, (V + 31) // 32))
    a.start = c.add(start, "start", torch.int32)
    a.tokens = c.add(tokens, "tokens", torch.int32)
    a.num_accepted = c.add(num_accepted, "num_accepted", torch.int32, shape=(B,))
    a.slots = c.add(slots, "slots", torch.int32, shape=(B,))
    a.dev_status = c.add(dev_status, "dev_status", _WORDS, at_least=1)
    return _finish(a, c)


def spec_count_tokens(count, stream=None):
    """Adds a batch's tokens to the table."""
    _launch(lib.spec_count_tokens, count, stream)


def adjust_args(target, target_out, cu_q, *, max_q_rows, draft=None, draft_out=None,
                draft_tokens=None, counts=None, seen=None, slots=None, repetition=1.0,
                presence=0.0, frequency=0.0, repetitions=None, presences=None, frequencies=None,
                bias_start=None, bias_tokens=None, bias_values=None, mask=None, mask_rows=None,
                ctx_tokens=None, dev_status=None):
    """sv_adjust_args for target [R, V] -> target_out (the same tensor: in
    place), optionally draft [R-B, V] -> draft_out, cu_q [B+1] int32 and
    draft_tokens [R-B] int32.  History: the table counts / seen with slots [B]
    int32, and ctx_tokens [n, B] int32 (tokens not yet in the table, such as
    the drafts so far at a draft position).  repetition / presence / frequency
    for all, or [B] float32 arrays.  Biases: entries bias_start[i] ..
    bias_start[i+1]-1 (int32 [B+1]) of bias_tokens (int32) and bias_values
    (float32).  Masks: mask [M, W] 32-bit words, W >= ceil(V / 32), bit 1 =
    allowed, with mask_rows [R] int32 (-1: none; None: row r takes mask r)."""
    a, c = AdjustArgs(), _Args()
    R, V = target.shape
    B = cu_q.shape[0] - 1
    floats = (torch.bfloat16, torch.float32)
    a.batch, a.vocab, a.max_q_rows, a.num_rows = B, V, int(max_q_rows), R
    a.target = c.add(target, "target", floats)
    a.dtype = _dt(target)
    a.target_out = c.add(target_out, "target_out", target.dtype, shape=(R, V))
    a.cu_q = c.add(cu_q, "cu_q", torch.int32)
    if draft is not None and draft.numel():
        a.draft = c.add(draft, "draft", target.dtype, shape=(R - B, V))
        if draft_out is None:
            raise ValueError("draft_out is None")
        a.draft_out = c.add(draft_out, "draft_out", target.dtype, shape=(R - B, V))
    if draft_tokens is not None and draft_tokens.numel():
        a.draft_tokens = c.add(draft_tokens, "draft_tokens", torch.int32, shape=(R - B,))
    if (counts is None) != (seen is None):
        raise ValueError("counts and seen go together")
    if counts is not None:
        a.num_slots = counts.shape[0]
        if a.num_slots < 1:
            raise ValueError("counts has no row")
        a.counts = c.add(counts, "counts", torch.int32, shape=(a.num_slots, V))
        a.seen = c.add(seen, "seen", _WORDS, shape=(a.num_slots, (V + 31) // 32))
        a.slots = c.add(slots, "slots", torch.int32, shape=(B,))
    if ctx_tokens is not None and ctx_tokens.numel():
        n, width = ctx_tokens.shape
        if width != B or (B > 1 and ctx_tokens.stride(1) != 1) or \
                (n > 1 and ctx_tokens.stride(0) < B):
            raise ValueError("ctx_tokens must be [n, B] with its rows contiguous")
        a.num_ctx, a.ctx_stride = n, ctx_tokens.stride(0) if n > 1 else B
        a.ctx_tokens = c.add(ctx_tokens, "ctx_tokens", torch.int32, rows=True)
    a.repetition, a.presence, a.frequency = float(repetition), float(presence), float(frequency)
    if not a.repetition > 0.0:
        raise ValueError("repetition must be > 0")
    a.repetitions = c.add(repetitions, "repetitions", torch.float32, shape=(B,))
    a.presences = c.add(presences, "presences", torch.float32, shape=(B,))
    a.frequencies = c.add(frequencies, "frequencies", torch.float32, shape=(B,))
    if bias_start is not None:
        if bias_tokens is None or bias_values is None:
            raise ValueError("bias_start needs bias_tokens and bias_values")
        a.num_bias = bias_tokens.numel()
        a.bias_start = c.add(bias_start, "bias_start", torch.int32, shape=(B + 1,))
        a.bias_tokens = c.add(bias_tokens, "bias_tokens", torch.int32)
        a.bias_values = c.add(bias_values, "bias_values", torch.float32, shape=(a.num_bias,))
    if mask is not None:
        a.num_masks, a.mask_stride = mask.shape
        a.mask = c.add(mask, "mask", _WORDS)
        a.mask_rows = c.add(mask_rows, "mask_rows", torch.int32, shape=(R,))
        if not a.mask:          # no rows: an empty tensor's null would mean no mask, whatever
            a.mask = a.cu_q     # rows mask_rows names (of num_masks = 0 rows none is read)
    a.dev_status = c.add(dev_status, "dev_status", _WORDS, at_least=1)
    return _finish(a, c)


def spec_adjust_logits(adjust, stream=None):
    """Penalties, biases and grammar masks on the target (and draft) rows."""
    _launch(lib.spec_adjust_logits, adjust, stream)
