"""Measured cases of the operators around a paged 4-bit KV cache, with their
plain forms.

The cache holds K and V as E2M1 codes (4 bits: 0, .5, 1, 1.5, 2, 3, 4, 6 and a
sign) with one E4M3 scale per 16 elements of a head and one factor per tensor, in
pages that a block table gives to sequences.  A token's rows of 128 elements take
72 bytes each for K and V, against 256 in bf16.

  norm_rope   RMS norm of every q and k head with the rotary positions in the same
              pass, to the contiguous rows that the unpaged attention takes
  append      a block's k and v (normed, rotated) as codes into their sequences'
              pages, q on the way; measured together with reading the rows back
  read        rows of the pages back as contiguous rows: a prefix handed to an
              unpaged cache, a request moved to another pool
  attn        attention of ragged block rows (a verify step) or single rows (a
              draft position, plain decoding) over the pages

`own` selects the package's kernels; otherwise `run` computes the plain form.
"""
import math

import numpy as np
import torch

own = False

_MOST8 = float(torch.finfo(torch.float8_e4m3fn).max)
_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_K_SCALE, _V_SCALE = 0.5, 0.25          # the cache's factors per tensor
_K_OUT, _V_OUT = 0.0625, 0.03125        # those of rows read back as E4M3 codes


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one draft position of the batch-8 workload: 8 single rows, 32 heads of 128
        _norm_rope("norm_draft_b8", B=8, r_lo=1, r_hi=1, Hq=32, Hkv=32),
        # verify block of the ragged GQA workload over an 8-bit cache, neighbouring pairs, half of
        # each head turned
        _norm_rope("norm_verify_gqa_b32", B=32, r_lo=2, r_hi=9, Hq=32, Hkv=8, layout="interleaved",
                   rot=64, kv="e4m3"),
        # prompts filling a cache, 32k rows, positions past the trained length
        _norm_rope("norm_prefill_32k", B=4, r_lo=8192, r_hi=8192, Hq=32, Hkv=8, scaling="yarn",
                   far=1 << 20),
        # one draft position entering the pages
        _append("append_draft_b8", B=8, r_lo=1, r_hi=1, Hq=32, Hkv=32, far=2048),
        # verify block of the large-vocabulary workload, normed, pages of 16
        _append("append_verify_b64", B=64, r_lo=9, r_hi=9, Hq=32, Hkv=8, norm=True, page=16, far=4096),
        # ragged prompts entering the pages, 17k rows
        _append("append_prompts_b3", B=3, r_lo=2731, r_hi=8192, Hq=32, Hkv=8, page=32,
                scaling="banded", far=1),
        # the shared prefix of the 32-sample workload handed to the unpaged pool
        _read("read_prefix_8k", B=1, r_lo=8192, r_hi=8192, Hkv=32, page=128),
        # ragged rows of the small workload's heads, fp32, an odd page size
        _read("read_f32_d64", B=7, r_lo=1, r_hi=700, Hkv=4, D=64, dtype="f32", page=48),
        # one draft position of the batch-8 workload: single rows over 512 to 2048 keys
        _attn("attn_draft_b8", B=8, r_lo=1, r_hi=1, Hq=32, Hkv=32, l_lo=512, l_hi=2048),
        # verify step of the ragged GQA workload: 2 to 9 rows over 128 to 8192 keys, pages of 16
        _attn("attn_verify_gqa_b32", B=32, r_lo=2, r_hi=9, Hq=32, Hkv=8, l_lo=128, l_hi=8192, page=16),
        # plain decoding at long context: four sequences of 128k keys
        _attn("attn_long_b4", B=4, r_lo=1, r_hi=1, Hq=32, Hkv=8, l_lo=131071, l_hi=131071),
        # the small workload's heads, lengths from nothing, an odd page size
        _attn("attn_odd_d64", B=13, r_lo=1, r_hi=5, Hq=4, Hkv=4, D=64, l_lo=0, l_hi=700, page=48),
    ]


def _norm_rope(name, B, r_lo, r_hi, Hq, Hkv, D=128, rot=0, layout="half", dtype="bf16", kv="",
               scaling="none", far=8192):
    return dict(name=name, op="norm_rope", B=B, r_lo=r_lo, r_hi=r_hi, Hq=Hq, Hkv=Hkv, D=D,
                rot=rot or D, layout=layout, dtype=dtype, kv=kv, scaling=scaling, l_lo=0, l_hi=far,
                norm=True)


def _append(name, B, r_lo, r_hi, Hq, Hkv, D=128, rot=0, layout="half", dtype="bf16", norm=False,
            page=64, scaling="none", far=8192):
    return dict(name=name, op="append", B=B, r_lo=r_lo, r_hi=r_hi, Hq=Hq, Hkv=Hkv, D=D, rot=rot or D,
                layout=layout, dtype=dtype, norm=norm, page=page, scaling=scaling, l_lo=0, l_hi=far)


def _read(name, B, r_lo, r_hi, Hkv, D=128, dtype="bf16", page=64):
    return dict(name=name, op="read", B=B, r_lo=r_lo, r_hi=r_hi, Hkv=Hkv, D=D, dtype=dtype, page=page,
                l_lo=0, l_hi=0)


def _attn(name, B, r_lo, r_hi, Hq, Hkv, l_lo, l_hi, D=128, page=64):
    return dict(name=name, op="attn", B=B, r_lo=r_lo, r_hi=r_hi, Hq=Hq, Hkv=Hkv, D=D, l_lo=l_lo,
                l_hi=l_hi, page=page)


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm_rope", "append", "read", "attn", "attn", "attn"))
    B = _log(rng, 1, 64)
    Hkv = rng.choice((1, 2, 4, 8))
    D = rng.choice((64, 128, 128))
    page = 16 * rng.choice((1, 2, 3, 4, 8))
    if op == "attn":
        g = rng.choice((1, 2, 4, 8))
        r = rng.randint(1, min(16, 64 // g))
        most = max(1, min(131072, (1 << 22) // (B * Hkv)))      # keys of all heads: the longest case's
        hi = _log(rng, 1, most)
        case = _attn("", B=B, r_lo=rng.randint(1, r), r_hi=r, Hq=Hkv * g, Hkv=Hkv, D=D,
                     l_lo=_log(rng, 1, hi) - 1, l_hi=hi - 1, page=page)
    else:
        rows = _log(rng, B, 16384)          # over the batch: single tokens to prompts
        r = max(1, rows // B)
        lo, dtype = max(1, r // 2), rng.choice(("bf16", "bf16", "f32"))
        if op == "read":
            case = _read("", B=B, r_lo=lo, r_hi=r, Hkv=Hkv, D=D, dtype=dtype, page=page)
        else:
            if op == "norm_rope":
                D = rng.choice((64, 96, 128, 128))
            how = dict(B=B, r_lo=lo, r_hi=r, Hq=Hkv * rng.choice((1, 2, 4)), Hkv=Hkv, D=D,
                       rot=2 * rng.randint(1, D // 2) if rng.random() < 0.4 else D,
                       layout=rng.choice(("half", "interleaved")), dtype=dtype,
                       scaling=rng.choice(("none", "linear", "ntk", "yarn", "banded")))
            if op == "norm_rope":
                case = _norm_rope("", kv=rng.choice(("", "", "e4m3")), far=_log(rng, 64, 1 << 24), **how)
            else:
                case = _append("", norm=rng.random() < 0.5, page=page, far=_log(rng, 1, 4096), **how)
    del case["name"]
    return case


# ---------------------------------------------------------------- inputs
def _spread(B, lo, hi):
    """Integers over [lo, hi], the same for every seed, so that a case's work is known from the
    case; over their logarithm where they span much."""
    step = (np.arange(B) * 0.6180339887498949 + 0.31) % 1.0
    if hi > 16 * max(lo, 1):
        n = np.floor(np.exp(np.log(max(lo, 1)) + step * (np.log(hi + 1) - np.log(max(lo, 1)))))
        n = np.where((n == 1) & (lo == 0) & (np.arange(B) % 2 == 1), 0, n)
    else:
        n = lo + np.floor(step * (hi - lo + 1))
    return np.clip(n, lo, hi).astype(np.int64)


def _rows(case):
    return _spread(case["B"], case["r_lo"], case["r_hi"])


def _lens(case):
    return _spread(case["B"], case["l_lo"], case["l_hi"])


def _cumulated(lens):
    cu = np.zeros(len(lens) + 1, dtype=np.int32)
    cu[1:] = np.cumsum(lens)
    return cu


def _torch_dtype(case):
    return torch.float32 if case.get("dtype") == "f32" else torch.bfloat16


def frequencies(rot, scaling, base=10000.0, factor=8.0, trained=8192):
    """Angle per token (radians) of the rot / 2 pairs in 64 bits, and the factor on cos and sin."""
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2.0))
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":               # pairs that turn often stay, slow ones are interpolated
        at = [rot * math.log(trained / (n * 2 * math.pi)) / (2 * math.log(base)) for n in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 0.001), 0.0, 1.0)
        return f / factor * ramp + f * (1.0 - ramp), 0.1 * math.log(factor) + 1.0
    if scaling == "banded":             # by the turns made over the trained length: below 1, above 4
        turns = trained * f / (2 * math.pi)
        keep = np.clip((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        return f / factor * (1.0 - keep) + f * keep, 1.0
    return f, 1.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    B, Hkv, D, R = case["B"], case["Hkv"], case["D"], int(_rows(case).sum())
    cu = _cumulated(_rows(case))
    dt = _torch_dtype(case)
    s = dict(case=case, cu_q=torch.from_numpy(cu).cuda(), max_rows=int(_rows(case).max()),
             kv_len=torch.from_numpy(_lens(case).astype(np.int32)).cuda(),
             status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if case["op"] in ("norm_rope", "append"):
        Hq = case["Hq"]
        if case["op"] == "norm_rope":   # positions anywhere below the farthest
            s["kv_len"] = torch.randint(0, case["l_hi"], (B,), generator=gen, device="cuda").to(torch.int32)
        qkv = torch.randn(R, Hq + 2 * Hkv, D, generator=gen, device="cuda").to(dt)
        f, mscale = frequencies(case["rot"], case["scaling"])
        turns = np.ldexp(f / (2 * math.pi), 64).astype(np.uint64)
        s.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], mscale=mscale,
                 f=torch.from_numpy(f).cuda(), turns=torch.from_numpy(turns.view(np.int64)).cuda(),
                 q_weight=None, k_weight=None, eps=1e-6,
                 q_out=torch.empty(R, Hq, D, dtype=dt, device="cuda"))
        if case["norm"]:
            s["q_weight"], s["k_weight"] = 1 + 0.2 * torch.randn(2, D, generator=gen, device="cuda")
    if case["op"] != "attn":
        kdt = torch.uint8 if case["op"] == "append" or case.get("kv") else dt
        s.update(k_out=torch.empty(R, Hkv, D, dtype=kdt, device="cuda"),
                 v_out=torch.empty(R, Hkv, D, dtype=kdt, device="cuda"))
    if case["op"] != "norm_rope":
        s["table"], s["num_pages"] = _table(case, gen)
        s["pages"] = _filled(case, s["num_pages"], gen)
    if case["op"] == "attn":
        s["q"] = torch.randn(R, case["Hq"], D, generator=gen, device="cuda").bfloat16()
        s["out"] = torch.empty_like(s["q"])
    return s


def _table(case, gen):
    """Pages of every sequence, scattered over a pool with some to spare; -1 behind the last."""
    need = -(-(_lens(case) + _rows(case)) // case["page"])
    num, start = int(need.sum()) + 5, torch.from_numpy(np.cumsum(need) - need).cuda()
    ids = torch.randperm(num, generator=gen, device="cuda").to(torch.int32)
    slot = torch.arange(int(need.max()), device="cuda")[None]
    return torch.where(slot < torch.from_numpy(need).cuda()[:, None],
                       ids[(start[:, None] + slot).clamp(max=num - 1)], -1), num


def _filled(case, num_pages, gen):
    """Pages [num_pages, Hkv, page / 16, 18 D] whose K and V are normal; a slab of 16 tokens is K's
    codes [16, D / 2], K's scales [16, D / 16], then the same of V."""
    Hkv, S, D = case["Hkv"], case["page"] // 16, case["D"]
    pages = torch.empty(num_pages, Hkv, S, 18 * D, dtype=torch.uint8, device="cuda")
    some = max(1, (1 << 25) // (Hkv * S * 16 * D))
    for p in range(0, num_pages, some):
        part = pages[p:p + some]
        for at, scale in ((0, _K_SCALE), (9 * D, _V_SCALE)):
            x = torch.randn(*part.shape[:3], 16, D, generator=gen, device="cuda")
            codes, scales = _quantized(x, scale)
            part[..., at:at + 8 * D] = _packed(codes).flatten(-2)
            part[..., at + 8 * D:at + 9 * D] = scales.view(torch.uint8).flatten(-2)
    return pages


def _quantized(x, factor):
    """Codes (0 .. 15) of fp32 values [.., D] and their scales [.., D / 16], E4M3."""
    y = x.unflatten(-1, (-1, 16))
    scales = (y.abs().amax(-1) / (6.0 * factor)).clamp(max=_MOST8).to(torch.float8_e4m3fn)
    unit = scales.float()[..., None] * factor
    q = torch.where(unit > 0, y / unit, torch.zeros_like(y))
    a = q.abs()
    code = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte()
            + (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5.0).byte())
    return (code + (torch.signbit(q).byte() << 3)).flatten(-2), scales


def _packed(codes):
    """Two codes to a byte, the even element's in the lower bits."""
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _values(codes, scales, factor):
    """fp32 values of packed codes [.., D / 2] with scales [.., D / 16] (bytes)."""
    grid = torch.tensor(_GRID + tuple(-g for g in _GRID), device=codes.device)
    both = torch.stack([grid[(codes & 15).int()], grid[(codes >> 4).int()]], dim=-1).flatten(-2)
    unit = scales.view(torch.float8_e4m3fn).float() * factor
    return (both.unflatten(-1, (-1, 16)) * unit[..., None]).flatten(-2)


# ---------------------------------------------------------------- one pass
def run(state):
    return {"norm_rope": _run_norm_rope, "append": _run_append, "read": _run_read,
            "attn": _run_attn}[state["case"]["op"]](state)


def _kept(state, build):
    """The package's call interface and the argument structs that a user's program keeps for these
    buffers (built once per set of buffers, as the step's other structs are)."""
    import speculative_decoding_verify_09_gb300 as pkg
    api = pkg.load()
    if "args" not in state:
        state["args"] = build(api)
    return api, state["args"]


def _cache(api, s):
    return api.Kv4Cache(s["num_pages"], s["case"]["Hkv"], s["case"]["D"], page_size=s["case"]["page"],
                        k_scale=_K_SCALE, v_scale=_V_SCALE, pages=s["pages"])


def _read_args(api, s, **scales):
    return api.kv4_read_args(_cache(api, s), s["table"], s["cu_q"], s["kv_len"], s["k_out"], s["v_out"],
                             max_q_rows=s["max_rows"], dev_status=s["status"], **scales)


def _positions(s, R):
    """Sequence and position of every row."""
    cu = s["cu_q"].long()
    seq = torch.repeat_interleave(torch.arange(s["case"]["B"], device="cuda"), cu[1:] - cu[:-1],
                                  output_size=R)
    return seq, s["kv_len"].long()[seq] + torch.arange(R, device="cuda") - cu[:-1][seq]


def _normed(x, weight, eps):
    y = x.float()
    if weight is None:
        return y
    return y * (y.square().mean(-1, keepdim=True) + eps).rsqrt() * weight


def _turned(y, pos, s):
    case, rot = s["case"], s["case"]["rot"]
    angle = pos.double()[:, None] * s["f"]
    cos = (angle.cos() * s["mscale"]).float()[:, None]
    sin = (angle.sin() * s["mscale"]).float()[:, None]
    if case["layout"] == "half":
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., rot:]], dim=-1)
    a, b = y[..., 0:rot:2], y[..., 1:rot:2]
    both = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([both.flatten(-2), y[..., rot:]], dim=-1)


def _as_e4m3(y, scale):
    return (y / scale).clamp(-_MOST8, _MOST8).to(torch.float8_e4m3fn)


def _run_norm_rope(s):
    case = s["case"]
    if own:
        api, args = _kept(s, lambda api: api.norm_rope_args(
            s["q"], s["k"], s["v"], s["q_out"], s["k_out"], s["v_out"], s["turns"],
            q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"], cu_q=s["cu_q"],
            kv_len=s["kv_len"], max_q_rows=s["max_rows"], layout=case["layout"], mscale=s["mscale"],
            k_scale=_K_OUT, v_scale=_V_OUT, dev_status=s["status"]))
        api.spec_norm_rope_rows(args)
        k, v = s["k_out"], s["v_out"]
        if case["kv"]:
            k, v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
        return s["q_out"], k, v
    _, pos = _positions(s, s["q"].shape[0])
    dt = s["q"].dtype
    q = _turned(_normed(s["q"], s["q_weight"], s["eps"]), pos, s).to(dt)
    k = _turned(_normed(s["k"], s["k_weight"], s["eps"]), pos, s)
    if case["kv"]:
        return q, _as_e4m3(k, _K_OUT), _as_e4m3(s["v"].float(), _V_OUT)
    return q, k.to(dt), s["v"].clone()


def _place(s, R):
    """Page, slab and token in the slab of every row."""
    page = s["case"]["page"]
    seq, pos = _positions(s, R)
    return s["table"].long()[seq, pos // page], pos % page // 16, pos % 16


def _run_append(s):
    case, D, R = s["case"], s["case"]["D"], s["q"].shape[0]
    if own:
        api, args = _kept(s, lambda api: (api.kv4_append_args(
            _cache(api, s), s["table"], s["cu_q"], s["kv_len"], s["k"], s["v"],
            max_q_rows=s["max_rows"], q=s["q"], q_out=s["q_out"], turns=s["turns"],
            q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"], layout=case["layout"],
            mscale=s["mscale"], dev_status=s["status"]),
            _read_args(api, s, k_scale=_K_OUT, v_scale=_V_OUT)))
        api.spec_kv4_append(args[0])
        api.spec_kv4_read(args[1])
        return s["q_out"], s["k_out"].view(torch.float8_e4m3fn), s["v_out"].view(torch.float8_e4m3fn)
    _, pos = _positions(s, R)
    q = _turned(_normed(s["q"], s["q_weight"], s["eps"]), pos, s).to(s["q"].dtype)
    k = _turned(_normed(s["k"], s["k_weight"], s["eps"]), pos, s)
    page, slab, t = _place(s, R)
    slabs = s["pages"].unflatten(-1, (2, 9 * D))
    codes, scales = slabs[..., :8 * D].unflatten(-1, (16, -1)), slabs[..., 8 * D:].unflatten(-1, (16, -1))
    out = []
    for n, (x, factor, to) in enumerate(((k, _K_SCALE, _K_OUT), (s["v"].float(), _V_SCALE, _V_OUT))):
        c, e = _quantized(x, factor)
        codes[page, :, slab, n, t] = _packed(c)
        scales[page, :, slab, n, t] = e.view(torch.uint8)
        out.append(_as_e4m3(_values(codes[page, :, slab, n, t], scales[page, :, slab, n, t], factor), to))
    return (q, *out)


def _run_read(s):
    D, R = s["case"]["D"], s["k_out"].shape[0]
    if own:
        api, args = _kept(s, lambda api: _read_args(api, s))
        api.spec_kv4_read(args)
        return s["k_out"], s["v_out"]
    page, slab, t = _place(s, R)
    slabs = s["pages"].unflatten(-1, (2, 9 * D))
    codes, scales = slabs[..., :8 * D].unflatten(-1, (16, -1)), slabs[..., 8 * D:].unflatten(-1, (16, -1))
    return tuple(_values(codes[page, :, slab, n, t], scales[page, :, slab, n, t], factor
                         ).to(s["k_out"].dtype) for n, factor in ((0, _K_SCALE), (1, _V_SCALE)))


def _run_attn(s):
    case = s["case"]
    if own:
        def build(api):
            args = api.kv4_attn_args(_cache(api, s), s["table"], s["cu_q"], s["kv_len"], s["q"], s["out"],
                                     max_q_rows=s["max_rows"], dev_status=s["status"])
            return args, api.kv4_workspace(args)
        api, args = _kept(s, build)
        api.spec_kv4_attn(*args)
        return s["out"]
    B, Hkv, D, page = case["B"], case["Hkv"], case["D"], case["page"]
    R, g, M = s["q"].shape[0], case["Hq"] // Hkv, s["max_rows"]
    slabs = s["pages"][s["table"].long().clamp(min=0)].transpose(1, 2).flatten(2, 3)  # [B, Hkv, slabs, 18 D]
    L = slabs.shape[2] * 16

    def values(at, factor):
        return _values(slabs[..., at:at + 8 * D].unflatten(-1, (16, -1)),
                       slabs[..., at + 8 * D:at + 9 * D].contiguous().unflatten(-1, (16, -1)),
                       factor).view(B, Hkv, L, D)

    cu = s["cu_q"].long()
    rows = cu[:-1, None] + torch.arange(M, device="cuda")            # [B, M], some behind their sequence
    q = s["q"][rows.clamp(max=R - 1)].float().view(B, M, Hkv, g, D).permute(0, 2, 1, 3, 4)
    score = q.reshape(B, Hkv, M * g, D) @ values(0, _K_SCALE).transpose(2, 3) * (1 / math.sqrt(D))
    last = s["kv_len"].long()[:, None] + torch.arange(M, device="cuda")          # a row's own position
    hidden = torch.arange(L, device="cuda") > last[..., None]                    # [B, M, L]
    score = score.view(B, Hkv, M, g, L).masked_fill(hidden[:, None, :, None], -math.inf)
    p = (score - score.amax(-1, keepdim=True)).exp()
    p = (p / p.sum(-1, keepdim=True)).view(B, Hkv, M * g, L)
    v = values(9 * D, _V_SCALE)
    # keys that no row sees may hold anything: a weight of zero does not undo an infinity
    v = v.masked_fill((torch.arange(L, device="cuda") >= (s["kv_len"].long() + cu[1:] - cu[:-1])[:, None])
                      [:, None, :, None], 0.0)
    out = (p @ v).view(B, Hkv, M, g, D).permute(0, 2, 1, 3, 4).reshape(B * M, Hkv * g, D)
    live = (rows < cu[1:, None]).flatten().nonzero_static(size=R)[:, 0]
    return out[live].to(s["q"].dtype)


# ---------------------------------------------------------------- floors
def work(case):
    B, Hkv, D = case["B"], case["Hkv"], case["D"]
    n = _rows(case)
    R, e = int(n.sum()), 4 if case.get("dtype") == "f32" else 2
    four = 2 * Hkv * D * (0.5 + 1 / 16)         # a token's K and V in the pages
    if case["op"] == "attn":
        keys = _lens(case) + n
        pairs = float((n * _lens(case) + n * (n + 1) / 2).sum())
        return {"bytes": float(keys.sum()) * four + 2 * R * case["Hq"] * D * 2 + 8 * B
                + 4 * float(np.ceil(keys / case["page"]).sum()), "flops": 4.0 * D * case["Hq"] * pairs}
    if case["op"] == "read":
        return {"bytes": R * (four + 2 * Hkv * D * e), "flops": 2.0 * R * 2 * Hkv * D}
    Hq = case["Hq"]
    flops = 7.0 * R * (Hq + Hkv) * D
    if case["op"] == "norm_rope":
        return {"bytes": R * D * (2 * Hq * e + 2 * Hkv * (e + (1 if case["kv"] else e))) + 8 * B,
                "flops": flops}
    # rows in, q out, the codes written and read again, their rows of E4M3 written
    return {"bytes": R * (D * (2 * Hq + 2 * Hkv) * e + 2 * four + 2 * Hkv * D) + 8 * B,
            "flops": flops + 6.0 * R * 2 * Hkv * D}


# ---------------------------------------------------------------- 64-bit values
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm_rope": _exact_rows, "append": _exact_rows, "read": _exact_read,
            "attn": _exact_attn}[case["op"]](s)


def _nearest(x, places):
    """Values of the grid (ascending, evenness by index) nearest to |x|, with x's sign."""
    grid = torch.tensor(places, dtype=torch.float64, device=x.device)
    a = x.abs().clamp(max=places[-1])
    hi = torch.searchsorted(grid, a.contiguous()).clamp(max=len(places) - 1)
    lo = (hi - 1).clamp(min=0)
    below, above = a - grid[lo], grid[hi] - a
    down = (below < above) | ((below == above) & (lo % 2 == 0))
    return torch.where(down, grid[lo], grid[hi]) * torch.where(x < 0, -1.0, 1.0).double()


_E4M3 = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
_E4M3 = _E4M3[:127]                     # up to 448; the last place is NaN


def _exact_rows(s):
    """Each pair (a, b) of a normed head as the complex number a + ib, turned by e^(i p f); what
    enters the pages, rounded twice: the scale, then the codes."""
    case = s["case"]
    rot, half = case["rot"], case["rot"] // 2
    cu, kv = s["cu_q"].cpu().numpy(), s["kv_len"].cpu().numpy().astype(np.int64)
    pos = np.concatenate([kv[i] + np.arange(cu[i + 1] - cu[i]) for i in range(case["B"])])
    f, mscale = frequencies(rot, case["scaling"])
    w = torch.from_numpy(mscale * np.exp(1j * (pos[:, None].astype(np.float64) * f[None]))).cuda()[:, None]
    out = []
    for name, weight, factor, to in (("q", s["q_weight"], 0, 0), ("k", s["k_weight"], _K_SCALE, _K_OUT),
                                     ("v", None, _V_SCALE, _V_OUT)):
        y = s[name].double().clone()
        if weight is not None:
            y /= torch.sqrt((y * y).sum(-1, keepdim=True) / case["D"] + s["eps"])
            y *= weight.double()
        if name != "v":
            if case["layout"] == "half":
                z = torch.complex(y[..., :half].contiguous(), y[..., half:rot].contiguous()) * w
                y[..., :half], y[..., half:rot] = z.real, z.imag
            else:
                z = torch.view_as_complex(y[..., :rot].unflatten(-1, (half, 2)).contiguous()) * w
                y[..., :rot] = torch.view_as_real(z).flatten(-2)
        if name != "q" and case["op"] == "append":
            b = y.unflatten(-1, (-1, 16))
            unit = _nearest(b.abs().amax(-1, keepdim=True) / (6 * factor), _E4M3) * factor
            y = (_nearest(b / unit.clamp(min=1e-300), _GRID) * unit).flatten(-2)
        if name != "q" and (case["op"] == "append" or case["kv"]):
            y = (y / to).clamp(-_MOST8, _MOST8)
        out.append(y)
    return tuple(out)


def _looked_up(rows, D, factor):
    """Rows of bytes [n, 16, D / 2] codes and [n, 16, D / 16] scales as float64 [16 n, D]."""
    codes, scales = rows
    one = np.array(_GRID + tuple(-g for g in _GRID))
    byte = torch.from_numpy(np.stack([one[np.arange(256) % 16], one[np.arange(256) // 16]], 1)).cuda()
    e4 = np.array(_E4M3 + [np.nan])
    e4 = torch.from_numpy(np.concatenate([e4, -e4]) * factor).cuda()
    x = byte[codes.reshape(-1, D // 2).long()].reshape(-1, D // 16, 16)
    return (x * e4[scales.reshape(-1, D // 16).long()][..., None]).reshape(-1, D)


def _sequence(s, i, h, at, factor):
    """K or V of sequence i, head h, from its first token on."""
    D = s["case"]["D"]
    ids = s["table"][i]
    slabs = s["pages"][ids[ids >= 0].long(), h].reshape(-1, 18 * D)
    return _looked_up((slabs[:, at:at + 8 * D], slabs[:, at + 8 * D:at + 9 * D]), D, factor)


def _exact_read(s):
    case, D, cu = s["case"], s["case"]["D"], s["cu_q"].tolist()
    return tuple(torch.cat([torch.stack([_sequence(s, i, h, at, factor)[:cu[i + 1] - cu[i]]
                                         for h in range(case["Hkv"])], 1) for i in range(case["B"])])
                 for at, factor in ((0, _K_SCALE), (9 * D, _V_SCALE)))


def _exact_attn(s):
    """Sequence by sequence, head by head, row by row."""
    case, D = s["case"], s["case"]["D"]
    g, cu, kv = case["Hq"] // case["Hkv"], s["cu_q"].tolist(), s["kv_len"].tolist()
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    for i in range(case["B"]):
        for h in range(case["Hkv"]):
            k, v = _sequence(s, i, h, 0, _K_SCALE), _sequence(s, i, h, 9 * D, _V_SCALE)
            for j in range(cu[i + 1] - cu[i]):
                n = kv[i] + j + 1
                q = s["q"][cu[i] + j, h * g:(h + 1) * g].double()
                e = torch.softmax(q @ k[:n].T / math.sqrt(D), dim=-1)
                out[cu[i] + j, h * g:(h + 1) * g] = e @ v[:n]
    return out
