"""Measured cases of the operators that stand around a verify step, with their
plain forms.

A verify step takes two things from the target's forward pass: the block rows'
q / k / v, which enter the attention and the KV cache, and the block's logits
rows, which enter the rejection sampler.  Three operators work on them:

  rope     rotary positions of ragged block rows (or of a prompt's rows): q and k
           rotated at their sequences' own positions, read from a fused
           projection's strided rows and written as the contiguous rows the
           attention takes; k and v optionally as E4M3 codes for an 8-bit cache
  adjust   repetition / presence / frequency penalties, biases and grammar masks
           on the target and draft rows, each row with the drafts before it
  count    the table of prompt and output tokens that the penalties read:
           filled from prompts, advanced by the tokens a verify step emits

`own` selects the package's kernels; otherwise `run` computes the plain form.
"""
import math

import numpy as np
import torch

own = False

_MOST = float(torch.finfo(torch.float8_e4m3fn).max)


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one draft position of the batch-8 workload: 8 single rows, 32 heads of 128
        _rope("rope_draft_b8", B=8, r_lo=1, r_hi=1, Hq=32, Hkv=32),
        # verify block of the ragged GQA workload, neighbouring-pair layout on half of each head
        _rope("rope_verify_gqa_b32", B=32, r_lo=2, r_hi=9, Hq=32, Hkv=8, layout="interleaved",
              rot=64),
        # verify block of the large-vocabulary workload over an 8-bit KV cache
        _rope("rope_verify_e4m3_b64", B=64, r_lo=9, r_hi=9, Hq=32, Hkv=8, kv="e4m3"),
        # prompts filling a cache, 32k rows, positions past the trained length
        _rope("rope_prefill_32k", B=4, r_lo=8192, r_hi=8192, Hq=32, Hkv=8, scaling="yarn",
              far=1 << 20),
        # fp32 rows of the small workload's heads, an odd count and an odd rotated part
        _rope("rope_f32_odd", B=61, r_lo=17, r_hi=17, Hq=4, Hkv=4, D=64, rot=20, dtype="f32"),
        # one draft position: single rows, the drafts so far as context
        _adjust("adjust_draft_b8", B=8, r_lo=1, r_hi=1, V=32000, ctx=3, draft=False),
        # verify step of the batch-8 workload, target and draft rows, half the rows with a grammar
        _adjust("adjust_verify_b8", B=8, r_lo=6, r_hi=6, V=32000, masked=0.5),
        # the largest: 576 target and 512 draft rows of 128256 tokens, not in place
        _adjust("adjust_verify_v128k_b64", B=64, r_lo=9, r_hi=9, V=128256, bias=64),
        # the same target rows in place, a quarter of them with a grammar
        _adjust("adjust_inplace_v128k_b64", B=64, r_lo=9, r_hi=9, V=128256, bias=64, masked=0.25,
                draft=False, inplace=True),
        # ragged fp32 rows of an odd vocabulary with everything on
        _adjust("adjust_f32_odd", B=13, r_lo=1, r_hi=5, V=32003, dtype="f32", bias=300, masked=0.5,
                ctx=1),
        # the tokens of one verify step entering the table
        _count("count_step_b64", B=64, n_lo=9, n_hi=9, V=128256, step=True),
        # 64 new requests: their slots cleared and their prompts counted
        _count("count_prompts_b64", B=64, n_lo=1024, n_hi=4096, V=128256, prompt=True, reset=True),
    ]


def _rope(name, B, r_lo, r_hi, Hq, Hkv, D=128, rot=0, layout="half", dtype="bf16", kv="",
          scaling="none", far=8192):
    return dict(name=name, op="rope", B=B, r_lo=r_lo, r_hi=r_hi, Hq=Hq, Hkv=Hkv, D=D, rot=rot or D,
                layout=layout, dtype=dtype, kv=kv, scaling=scaling, far=far)


def _adjust(name, B, r_lo, r_hi, V, dtype="bf16", hist=2048, bias=0, masked=0.0, ctx=0, draft=True,
            inplace=False):
    return dict(name=name, op="adjust", B=B, r_lo=r_lo, r_hi=r_hi, V=V, dtype=dtype, hist=hist,
                bias=bias, masked=masked, ctx=ctx, draft=draft, inplace=inplace)


def _count(name, B, n_lo, n_hi, V, step=False, prompt=False, reset=False):
    return dict(name=name, op="count", B=B, n_lo=n_lo, n_hi=n_hi, V=V, step=step, prompt=prompt,
                reset=reset)


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "rope", "adjust", "adjust", "count"))
    B = _log(rng, 1, 64)
    if op == "rope":
        D = rng.choice((64, 128))
        Hkv = rng.choice((1, 2, 4, 8))
        rows = _log(rng, B, 16384)          # over the batch: single tokens to prompts
        r = max(1, rows // B)
        case = _rope("", B=B, r_lo=max(1, r // 2), r_hi=r, Hq=Hkv * rng.choice((1, 2, 4)), Hkv=Hkv,
                     D=D, rot=2 * rng.randint(1, D // 2) if rng.random() < 0.4 else D,
                     layout=rng.choice(("half", "interleaved")),
                     dtype=rng.choice(("bf16", "bf16", "f32")),
                     scaling=rng.choice(("none", "linear", "ntk", "yarn", "banded")),
                     far=_log(rng, 64, 1 << 24))
        if case["dtype"] == "bf16" and rng.random() < 0.4:
            case["kv"] = "e4m3"
    elif op == "adjust":
        r = rng.randint(1, 9)
        V = _log(rng, 100, 128256)
        case = _adjust("", B=B, r_lo=rng.randint(1, r), r_hi=r, V=V,
                       dtype=rng.choice(("bf16", "bf16", "f32")) if B < 32 else "bf16",
                       hist=_log(rng, 1, 8192), bias=rng.choice((0, 1, rng.randint(2, 400))),
                       masked=rng.choice((0.0, 0.3, 1.0)), ctx=rng.randint(0, 5),
                       draft=rng.random() < 0.6, inplace=rng.random() < 0.4)
    else:
        prompt = rng.random() < 0.5
        n = _log(rng, 1, 4096)
        case = _count("", B=B, n_lo=rng.randint(0, n), n_hi=n, V=_log(rng, 100, 128256),
                      prompt=prompt, reset=rng.random() < 0.5, step=not prompt and n <= 16)
    del case["name"]
    return case


# ---------------------------------------------------------------- inputs
def _lens(case, lo, hi):
    """Rows (or tokens) of each sequence: spread over [lo, hi], the same for every seed, so
    that a case's work is known from the case."""
    B = case["B"]
    step = (np.arange(B) * 0.6180339887498949) % 1.0
    return np.minimum(hi, lo + np.floor(step * (hi - lo + 1)).astype(np.int64))


def _torch_dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _cumulated(lens):
    cu = np.zeros(len(lens) + 1, dtype=np.int32)
    cu[1:] = np.cumsum(lens)
    return cu


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


def _tokens(gen, shape, V):
    """Token ids as text has them: a few very frequent, most rare."""
    u = torch.rand(shape, generator=gen, device="cuda", dtype=torch.float64)
    return (u.pow(3) * V).to(torch.int32).clamp_(0, V - 1)


def _bits(truth):
    """Truth values [n, V] as 32-bit words [n, ceil(V / 32)], token t at bit t % 32 of word t / 32."""
    n, V = truth.shape
    W = (V + 31) // 32
    t = torch.zeros(n, W * 32, dtype=torch.int64, device=truth.device)
    t[:, :V] = truth
    w = (t.view(n, W, 32) << torch.arange(32, device=truth.device)).sum(2)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    return {"rope": _prepare_rope, "adjust": _prepare_adjust, "count": _prepare_count}[case["op"]](
        case, gen)


def _prepare_rope(case, gen):
    lens = _lens(case, case["r_lo"], case["r_hi"])
    cu = _cumulated(lens)
    R, Hq, Hkv, D = int(cu[-1]), case["Hq"], case["Hkv"], case["D"]
    dt = _torch_dtype(case)
    qkv = torch.randn(R, Hq + 2 * Hkv, D, generator=gen, device="cuda").to(dt)
    f, mscale = frequencies(case["rot"], case["scaling"])
    turns = np.ldexp(f / (2 * math.pi), 64).astype(np.uint64)
    kv_len = torch.randint(0, case["far"], (case["B"],), generator=gen, device="cuda").to(torch.int32)
    kdt = torch.uint8 if case["kv"] else dt
    return dict(case=case, q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:],
                cu_q=torch.from_numpy(cu).cuda(), kv_len=kv_len,
                f=torch.from_numpy(f).cuda(), turns=torch.from_numpy(turns.view(np.int64)).cuda(),
                mscale=mscale, k_scale=0.0625, v_scale=0.0625, max_rows=int(lens.max()),
                q_out=torch.empty(R, Hq, D, dtype=dt, device="cuda"),
                k_out=torch.empty(R, Hkv, D, dtype=kdt, device="cuda"),
                v_out=torch.empty(R, Hkv, D, dtype=kdt, device="cuda"),
                status=torch.zeros(1, dtype=torch.int32, device="cuda"))


def _prepare_adjust(case, gen):
    B, V = case["B"], case["V"]
    lens = _lens(case, case["r_lo"], case["r_hi"])
    cu = _cumulated(lens)
    R, dt = int(cu[-1]), _torch_dtype(case)
    s = dict(case=case, cu_q=torch.from_numpy(cu).cuda(), max_rows=int(lens.max()),
             target=(torch.randn(R, V, generator=gen, device="cuda") * 3).to(dt),
             draft_tokens=_tokens(gen, (R - B,), V), draft=None, draft_out=None,
             status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    s["target_out"] = s["target"] if case["inplace"] else torch.empty_like(s["target"])
    if case["draft"] and R > B:
        s["draft"] = (torch.randn(R - B, V, generator=gen, device="cuda") * 3).to(dt)
        s["draft_out"] = s["draft"] if case["inplace"] else torch.empty_like(s["draft"])
    # history: three quarters prompt, one quarter output, in slots of a larger table
    S, n = B + 3, case["hist"]
    slots = torch.randperm(S, generator=gen, device="cuda")[:B].to(torch.int32)
    hist = _tokens(gen, (B, n), V).long()
    cut = n - n // 4
    counts = torch.zeros(S, V, dtype=torch.int32, device="cuda")
    at = slots.long()[:, None].expand(B, n)
    counts.index_put_((at[:, cut:], hist[:, cut:]),
                      torch.ones(B, n - cut, dtype=torch.int32, device="cuda"), accumulate=True)
    prompt = torch.zeros(S, V, dtype=torch.bool, device="cuda")
    prompt[at[:, :cut], hist[:, :cut]] = True
    counts |= prompt.to(torch.int32) << 31           # the sign bit marks prompt tokens
    s.update(slots=slots, counts=counts, seen=_bits(counts != 0))

    def spread(lo, hi):
        return torch.rand(B, generator=gen, device="cuda") * (hi - lo) + lo

    s.update(repetitions=spread(1.0, 1.5), presences=spread(0.0, 0.8), frequencies=spread(0.0, 0.5))
    s.update(bias_start=None, bias_tokens=None, bias_values=None, mask=None, mask_rows=None, ctx=None)
    if case["bias"]:
        # distinct tokens per sequence, as the keys of a request's bias table are
        nb = min(case["bias"], V)
        pick = torch.randint(0, V, (B, 1), generator=gen, device="cuda")
        s.update(bias_start=torch.arange(B + 1, device="cuda", dtype=torch.int32) * nb,
                 bias_tokens=((pick + torch.arange(nb, device="cuda") * (V // nb)) % V
                              ).to(torch.int32).reshape(-1),
                 bias_values=torch.randn(B * nb, generator=gen, device="cuda") * 4)
    if case["masked"]:
        # a grammar allows few tokens (a keyword) or most (inside a string)
        m = int(case["masked"] * R)
        share = torch.where(torch.arange(m, device="cuda") % 2 == 0, 0.01, 0.9)
        s["mask"] = _bits(torch.rand(m, V, generator=gen, device="cuda") < share[:, None])
        s["mask_rows"] = torch.full((R,), -1, dtype=torch.int32, device="cuda")
        s["mask_rows"][torch.randperm(R, generator=gen, device="cuda")[:m]] = \
            torch.arange(m, device="cuda", dtype=torch.int32)
    if case["ctx"]:
        s["ctx"] = _tokens(gen, (case["ctx"], B), V)
    return s


def _prepare_count(case, gen):
    B, V = case["B"], case["V"]
    start = _cumulated(_lens(case, case["n_lo"], case["n_hi"]))
    T, S = int(start[-1]), B + 3
    s = dict(case=case, tokens=_tokens(gen, (T,), V), start=torch.from_numpy(start).cuda(),
             slots=torch.randperm(S, generator=gen, device="cuda")[:B].to(torch.int32),
             accepted=None, status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if case["step"]:
        n = torch.from_numpy(np.diff(start)).cuda()
        u = torch.rand(B, generator=gen, device="cuda")
        s["accepted"] = (u * n).floor().to(torch.int32).minimum(n - 1)   # -1 where n is 0
    counts = torch.zeros(S, V, dtype=torch.int32, device="cuda")
    old = _tokens(gen, (S, 512), V).long()
    counts.scatter_add_(1, old, torch.ones_like(old, dtype=torch.int32))
    s.update(counts=counts, seen=_bits(counts != 0))
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    return {"rope": _run_rope, "adjust": _run_adjust, "count": _run_count}[state["case"]["op"]](state)


def _api(state, build):
    """The package's call interface and the argument struct that a user's program keeps for these
    buffers (built once per set of buffers, as the step's other structs are)."""
    import speculative_decoding_verify_09_gb300 as pkg
    api = pkg.load()
    if "args" not in state:
        state["args"] = build(api)
    return api, state["args"]


def _sequence_of_rows(cu, R):
    B = cu.shape[0] - 1
    seq = torch.repeat_interleave(torch.arange(B, device=cu.device), (cu[1:] - cu[:-1]).long(),
                                  output_size=R)
    return seq, torch.arange(R, device=cu.device) - cu[:-1].long()[seq]


def _run_rope(s):
    case = s["case"]
    if own:
        api, args = _api(s, lambda api: api.rope_args(
            s["q"], s["k"], s["v"], s["q_out"], s["k_out"], s["v_out"], s["turns"],
            cu_q=s["cu_q"], kv_len=s["kv_len"], max_q_rows=s["max_rows"], layout=case["layout"],
            mscale=s["mscale"], k_scale=s["k_scale"], v_scale=s["v_scale"],
            dev_status=s["status"]))
        api.spec_rope_rows(args)
        k, v = s["k_out"], s["v_out"]
        if case["kv"]:
            k, v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
        return s["q_out"], k, v
    R, rot = s["q"].shape[0], case["rot"]
    seq, j = _sequence_of_rows(s["cu_q"], R)
    angle = (s["kv_len"].long()[seq] + j).double()[:, None] * s["f"]
    cos = (angle.cos() * s["mscale"]).float()[:, None]
    sin = (angle.sin() * s["mscale"]).float()[:, None]

    def turn(x):
        y = x.float()
        if case["layout"] == "half":
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            return torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., rot:]], dim=-1)
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        both = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1)
        return torch.cat([both.flatten(-2), y[..., rot:]], dim=-1)

    def cached(y, scale):
        if not case["kv"]:
            return y.to(s["q"].dtype)
        return (y / scale).clamp(-_MOST, _MOST).to(torch.float8_e4m3fn)

    return (turn(s["q"]).to(s["q"].dtype), cached(turn(s["k"]), s["k_scale"]),
            cached(s["v"].float(), s["v_scale"]))


def _run_adjust(s):
    case = s["case"]
    B, V = case["B"], case["V"]
    if own:
        api, args = _api(s, lambda api: api.adjust_args(
            s["target"], s["target_out"], s["cu_q"], max_q_rows=s["max_rows"], draft=s["draft"],
            draft_out=s["draft_out"], draft_tokens=s["draft_tokens"], counts=s["counts"],
            seen=s["seen"], slots=s["slots"], repetitions=s["repetitions"],
            presences=s["presences"], frequencies=s["frequencies"], bias_start=s["bias_start"],
            bias_tokens=s["bias_tokens"], bias_values=s["bias_values"], mask=s["mask"],
            mask_rows=s["mask_rows"], ctx_tokens=s["ctx"], dev_status=s["status"]))
        api.spec_adjust_logits(args)
        return (s["target_out"],) if s["draft"] is None else (s["target_out"], s["draft_out"])
    R = s["target"].shape[0]
    seq, j = _sequence_of_rows(s["cu_q"], R)
    c = s["counts"][s["slots"].long()][seq]                     # [R, V]
    prompt, n = c < 0, c & 0x7FFFFFFF
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    if s["ctx"] is not None:
        rows = torch.arange(R, device="cuda")[None].expand(case["ctx"], R)
        n.index_put_((rows, s["ctx"].long()[:, seq]), one, accumulate=True)
    # row j of a sequence has its drafts 1 .. j behind it: every (row, draft) pair, the later
    # drafts with weight zero
    if R > B:
        b = torch.arange(s["max_rows"], device="cuda")[None].expand(R, s["max_rows"])
        rows = torch.arange(R, device="cuda")[:, None].expand_as(b)
        first = (s["cu_q"][:-1].long() - torch.arange(B, device="cuda"))[seq]
        at = (first[:, None] + b).clamp(max=R - B - 1)
        n.index_put_((rows, s["draft_tokens"].long()[at]), (b < j[:, None]).to(torch.int32),
                     accumulate=True)
    used = n > 0
    rep, pres, freq = (s[k][seq][:, None] for k in ("repetitions", "presences", "frequencies"))
    less = n.float() * freq + used.float() * pres
    known = prompt | used
    bias = None
    if s["bias_start"] is not None:
        nb = s["bias_tokens"].numel() // B
        bias = torch.zeros(B, V, device="cuda").scatter_(1, s["bias_tokens"].long().view(B, nb),
                                                         s["bias_values"].view(B, nb))[seq]
    barred = None
    if s["mask"] is not None:
        w = s["mask"][s["mask_rows"].long().clamp(min=0)]
        allowed = ((w[:, :, None] >> torch.arange(32, device="cuda")) & 1).flatten(1)[:, :V] != 0
        barred = ~allowed & (s["mask_rows"] >= 0)[:, None]

    def adjusted(x, rows):
        y = x.float()
        r = rep if rows is None else rep[rows]
        y = torch.where(known if rows is None else known[rows],
                        torch.where(y > 0, y / r, y * r), y)
        y = y - (less if rows is None else less[rows])
        if bias is not None:
            y = y + (bias if rows is None else bias[rows])
        if barred is not None:
            y = y.masked_fill(barred if rows is None else barred[rows], -math.inf)
        return y.to(x.dtype)

    out = [adjusted(s["target"], None)]
    if s["draft"] is not None:          # draft row j has the context of target row j
        last = s["cu_q"][1:].long() - 1
        is_last = torch.zeros(R, dtype=torch.bool, device="cuda").index_fill_(0, last, True)
        rows = (~is_last).nonzero_static(size=R - B)[:, 0]
        out.append(adjusted(s["draft"], rows))
    if case["inplace"]:
        out = [x.copy_(y) for x, y in zip((s["target"], s["draft"]), out)]
    return tuple(out)


def _run_count(s):
    case = s["case"]
    if own:
        api, args = _api(s, lambda api: api.count_args(
            s["counts"], s["seen"], s["tokens"], s["start"], slots=s["slots"],
            num_accepted=s["accepted"], prompt=case["prompt"], reset=case["reset"],
            dev_status=s["status"]))
        api.spec_count_tokens(args)
        return s["counts"], s["seen"]
    slots, T = s["slots"].long(), s["tokens"].shape[0]
    if case["reset"]:
        s["counts"].index_fill_(0, slots, 0)
    seq, j = _sequence_of_rows(s["start"], T)
    tokens = s["tokens"].long()
    take = torch.ones(T, dtype=torch.int32, device="cuda")
    if s["accepted"] is not None:
        take = (j <= s["accepted"].long()[seq]).to(torch.int32)
    if case["prompt"]:
        mark = torch.zeros_like(s["counts"])
        mark.index_put_((slots[seq], tokens), take, accumulate=True)
        s["counts"] |= (mark > 0).to(torch.int32) << 31
    else:
        s["counts"].index_put_((slots[seq], tokens), take, accumulate=True)
    s["seen"].copy_(_bits(s["counts"] != 0))
    return s["counts"], s["seen"]


# ---------------------------------------------------------------- floors
def _distinct(n, V):
    """Expected number of distinct tokens among n of `_tokens`."""
    edge = (np.arange(V + 1) / V) ** (1.0 / 3.0)
    return float(-np.expm1(n * np.log1p(-np.minimum(np.diff(edge), 1 - 1e-12))).sum())


def work(case):
    B = case["B"]
    if case["op"] == "rope":
        R = int(_lens(case, case["r_lo"], case["r_hi"]).sum())
        e = 2 if case["dtype"] == "bf16" else 4
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        moved = R * D * (2 * Hq * e + 2 * Hkv * (e + (1 if case["kv"] else e)))
        return {"bytes": moved + 8 * B, "flops": 3.0 * R * (Hq + Hkv) * case["rot"]}
    V, W = case["V"], (case["V"] + 31) // 32
    if case["op"] == "count":
        n = _lens(case, case["n_lo"], case["n_hi"])
        new = sum(_distinct(int(x), V) for x in n)
        moved = 4.0 * n.sum() + 8 * new + 12 * B
        if case["reset"]:       # the old entries cleared, found by the table's bits
            moved += B * (4 * W + 4 * _distinct(512, V))
        return {"bytes": moved, "flops": float(n.sum())}
    e = 2 if case["dtype"] == "bf16" else 4
    R = int(_lens(case, case["r_lo"], case["r_hi"]).sum())
    m = int(case["masked"] * R)
    both = 2 if case["draft"] else 1
    rows = both * R - (B if case["draft"] else 0)
    known = _distinct(case["hist"], V)
    touched = min(V, known + min(case["bias"], V))
    moved = B * (4 * W + 4 * known + 8 * min(case["bias"], V)) + m * 4 * W
    if case["inplace"]:         # barred tokens are written; the others only where something changes
        barred = m * (0.99 + 0.1) / 2 * V
        moved += both * barred * e + rows * touched * 2 * e
    else:
        moved += rows * V * 2 * e
    return {"bytes": moved, "flops": 6.0 * rows * touched}


# ---------------------------------------------------------------- 64-bit values
def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "adjust": _exact_adjust, "count": _exact_count}[case["op"]](s)


def _exact_rope(s):
    """Each pair (a, b) as the complex number a + ib, turned by e^(i p f)."""
    case = s["case"]
    rot, half = case["rot"], case["rot"] // 2
    cu, kv = s["cu_q"].cpu().numpy(), s["kv_len"].cpu().numpy().astype(np.int64)
    pos = np.concatenate([kv[i] + np.arange(cu[i + 1] - cu[i]) for i in range(case["B"])])
    f, mscale = frequencies(rot, case["scaling"])
    angle = pos[:, None].astype(np.float64) * f[None]
    w = torch.from_numpy(mscale * np.exp(1j * angle)).cuda()[:, None]
    out = []
    for name, scale in (("q", 0.0), ("k", s["k_scale"]), ("v", s["v_scale"])):
        y = s[name].double().clone()
        if name != "v":
            if case["layout"] == "half":
                z = torch.complex(y[..., :half].contiguous(), y[..., half:rot].contiguous()) * w
                y[..., :half], y[..., half:rot] = z.real, z.imag
            else:
                z = torch.view_as_complex(y[..., :rot].unflatten(-1, (half, 2)).contiguous()) * w
                y[..., :rot] = torch.view_as_real(z).flatten(-2)
        if case["kv"] and scale:
            y = (y / scale).clamp(-_MOST, _MOST)
        out.append(y)
    return tuple(out)


def _exact_adjust(s):
    """Sequence by sequence, row by row, the context carried along."""
    case, V = s["case"], s["case"]["V"]
    cu = s["cu_q"].tolist()
    slots, tokens = s["slots"].tolist(), s["draft_tokens"].tolist()
    at = s["mask_rows"].tolist() if s["mask_rows"] is not None else None
    pos = torch.arange(V, device="cuda")
    outs = [s["target"].double()]
    if s["draft"] is not None:
        outs.append(s["draft"].double())
    for i in range(case["B"]):
        word = s["counts"][slots[i]].to(torch.int64)
        prompt = word < 0
        n = torch.where(prompt, word + (1 << 31), word)
        if s["ctx"] is not None:
            for t in s["ctx"][:, i].tolist():
                n[t] += 1
        rep, pres, freq = (float(s[k][i]) for k in ("repetitions", "presences", "frequencies"))
        add = torch.zeros(V, dtype=torch.float64, device="cuda")
        if s["bias_start"] is not None:
            lo, hi = int(s["bias_start"][i]), int(s["bias_start"][i + 1])
            add[s["bias_tokens"][lo:hi].long()] = s["bias_values"][lo:hi].double()
        for j in range(cu[i + 1] - cu[i]):
            r = cu[i] + j
            if j:
                n[tokens[r - i - 1]] += 1
            rows = [(outs[0], r)]
            if len(outs) > 1 and r + 1 < cu[i + 1]:     # the bonus row has no draft row
                rows.append((outs[1], r - i))
            for x, row in rows:
                y = x[row]
                factor = torch.where(y > 0, 1.0 / rep, rep)
                y *= torch.where(prompt | (n > 0), factor, 1.0)
                y -= freq * n + pres * (n > 0)
                y += add
                if at is not None and at[r] >= 0:
                    w = s["mask"][at[r]].to(torch.int64) & 0xFFFFFFFF
                    y[((w[pos // 32] >> (pos % 32)) & 1) == 0] = -math.inf
    return tuple(outs)


def _exact_count(s):
    case, V = s["case"], s["case"]["V"]
    counts = s["counts"].cpu().numpy().view(np.uint32).astype(np.int64)
    slots, start = s["slots"].tolist(), s["start"].tolist()
    tokens = s["tokens"].cpu().numpy()
    kept = s["accepted"].tolist() if s["accepted"] is not None else None
    if case["reset"]:
        counts[slots] = 0
    for i, slot in enumerate(slots):
        hi = start[i + 1] if kept is None else start[i] + kept[i] + 1
        mine = tokens[start[i]:hi]
        if case["prompt"]:
            counts[slot, mine] |= 1 << 31
        else:
            counts[slot] += np.bincount(mine, minlength=V)
    pad = np.zeros((counts.shape[0], (V + 31) // 32 * 32), dtype=bool)
    pad[:, :V] = counts != 0
    seen = np.packbits(pad, axis=1, bitorder="little").view("<u4").astype(np.uint32).view(np.int32)
    return counts.astype(np.uint32).view(np.int32), seen
