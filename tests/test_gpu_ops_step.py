"""The operators in the order a serving loop uses them, over several steps:
rotary positions of the block rows, draft positions on adjusted logits, the
adjusted verify step, and its tokens into the table.  Each operator's output is
compared with the float64 oracle's on the inputs it really had (the device's
bits of the step before it), so every comparison is as strict as the operator's
own: tokens, lengths and cache rows exactly outside the near-tie windows."""
import numpy as np
import pytest
import torch

import oracle
import workloads as W
from gpu_util import DeviceStep, compare_sampling, dev, host_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    import speculative_decoding_verify_09_gb300 as pkg
    pkg.build()
    return pkg.load()


def _near(got_bits, want, slack):
    """bf16 within half a step plus `slack` of the float64 value."""
    got = oracle.to_f64(got_bits)
    fin = np.isfinite(want)
    assert np.array_equal(got[~fin], want[~fin])
    assert np.all(np.abs(got[fin] - want[fin]) <= 2.0 ** -8 * np.abs(want[fin]) + slack)


@pytest.mark.parametrize("kv", ["", "e4m3"])
def test_steps_of_a_serving_loop(api, kv):
    B, K, V, D, steps = 3, 4, 2003, 128, 3
    base = W.workload("bass_b8", B=B, V=V, Hq=2, Hkv=2, L_lo=20, L_hi=90, K_fixed=(K,) * B,
                      cap_slack=steps * (K + 2), kv_dtype=kv, temperature=0.8, gen_seed=40)
    rng = np.random.default_rng(41)
    turns, m = api.rope_turns(64, scaling="yarn", factor=4.0, trained_len=64)
    freqs, m64 = oracle.rope_frequencies(64, kind="yarn", factor=4.0, trained=64)

    # the requests enter: prompts into the table, in slots of their own
    table = api.TokenCounts(B + 2, V)
    ref = np.zeros((B + 2, V), dtype=np.int32)
    slots = np.array([3, 0, 4], np.int32)
    start = np.array([0, 30, 55, 100], np.int32)
    prompt = rng.integers(0, V // 4, 100).astype(np.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.spec_count_tokens(api.count_args(table.counts, table.seen, dev(prompt), dev(start),
                                         slots=dev(slots), prompt=True, reset=True,
                                         dev_status=status))
    ref, _, _ = oracle.count_tokens(ref, prompt, start, slots=slots, prompt=True, reset=True)
    pen = dict(repetition=np.array([1.2, 1.0, 0.9], np.float32),
               presence=np.array([0.3, 0.0, 0.1], np.float32),
               frequency=np.array([0.2, 0.5, 0.0], np.float32))
    args = dict(repetitions=dev(pen["repetition"]), presences=dev(pen["presence"]),
                frequencies=dev(pen["frequency"]), slots=dev(slots), counts=table.counts,
                seen=table.seen, dev_status=status)
    slack = 5 * 2.0 ** -24 * 40

    inp = W.make_inputs(base)
    for step in range(steps):
        if step:                        # new rows of a new forward pass, the caches go on
            fresh = W.make_inputs(W.workload("bass_b8", B=B, V=V, Hq=2, Hkv=2, L_lo=20, L_hi=90,
                                             K_fixed=(K,) * B, kv_dtype=kv, gen_seed=50 + step))
            for k in ("q", "target_logits", "draft_logits", "k_new", "v_new"):
                inp[k] = fresh[k]
        cu, kv_len = inp["cu_q"], inp["kv_len"]
        R = int(cu[-1])
        # 1. rotary positions, out of one fused projection, into the cache's format
        qkv = W.f32_to_bf16_bits(rng.standard_normal((R, 6, D), dtype=np.float32))
        d = DeviceStep(inp, api)
        x = dev(qkv)
        api.spec_rope_rows(api.rope_args(x[:, :2], x[:, 2:4], x[:, 4:], d.q, d.k_new, d.v_new, turns,
                                         cu_q=d.cu_q, kv_len=d.kv_len, max_q_rows=d.max_q_rows,
                                         mscale=m, k_scale=inp.get("k_scale", 0.0),
                                         v_scale=inp.get("v_scale", 0.0), dev_status=status))
        torch.cuda.synchronize()
        pos = oracle.row_positions(cu, kv_len)
        x64 = oracle.to_f64(qkv)
        wq, wk = (oracle.rope_rows(x64[:, h], pos, freqs, "half", m64)
                  for h in (slice(0, 2), slice(2, 4)))
        _near(host_bits(d.q), wq, 1e-5 * m64)
        if kv:
            for t, w in ((d.k_new, wk), (d.v_new, x64[:, 4:])):
                y = np.clip(w / inp["k_scale"], -448, 448)
                best = np.abs(oracle.to_f64(oracle.e4m3_nearest(y)) - y)
                got = oracle.to_f64(t.cpu().numpy())
                assert np.all(np.abs(got - y) <= best + 4e-5 * m64 / inp["k_scale"])
        else:
            _near(host_bits(d.k_new), wk, 1e-5 * m64)
            assert np.array_equal(host_bits(d.v_new), qkv[:, 4:])
        inp["q"], inp["k_new"], inp["v_new"] = (host_bits(t) for t in (d.q, d.k_new, d.v_new))

        # 2. draft positions: adjusted draft rows with the drafts so far, and their draws
        mask = np.full((R, (V + 31) // 32), -1, dtype=np.int32)
        mask[:, :8] = rng.integers(-2 ** 31, 2 ** 31, (R, 8))
        rows = np.where(rng.random(R) < 0.5, np.arange(R), -1).astype(np.int32)
        at = np.arange(B)
        raw = inp["draft_logits"].reshape(B, K, V)
        adjusted = torch.empty(B, K, V, dtype=torch.bfloat16, device="cuda")
        drafts = torch.zeros(K, B, dtype=torch.int32, device="cuda")
        for t in range(K):
            line = dev(np.ascontiguousarray(raw[:, t]))
            here = np.ascontiguousarray(rows[cu[:-1] + t])
            api.spec_adjust_logits(api.adjust_args(
                line, line, dev(np.arange(B + 1, dtype=np.int32)), max_q_rows=1,
                ctx_tokens=drafts[:t], mask=dev(mask), mask_rows=dev(here), **args))
            lens = dev((kv_len + t).astype(np.int32))
            a = api.draft_args(line, lens, drafts[t], temperature=0.8, top_p=1.0, seed=7,
                               seq_ids=d.seq_ids, dev_status=status)
            api.spec_draft_sample(a, api.Workspace(api.draft_workspace_bytes(a)))
            adjusted[:, t] = line
            torch.cuda.synchronize()
            want, _, _ = oracle.adjust_logits(
                np.ascontiguousarray(raw[:, t]), np.arange(B + 1), counts=ref, slots=slots,
                ctx=drafts[:t].cpu().numpy(), mask=mask, mask_rows=here, **pen)
            _near(host_bits(line), want, slack)
            got = oracle.draft_sample(host_bits(line), kv_len + t, 0.8, 1.0, 7, inp["seq_ids"])
            tok, tied = got["tokens"], got["tie"]
            assert all(tied[i] or int(drafts[t, i]) == int(tok[i]) for i in at), t
        tokens = np.ascontiguousarray(drafts.t().cpu().numpy()).reshape(-1)

        # 3. the verify step on adjusted target rows and the adjusted draft rows as drawn from
        d.drafts.copy_(dev(tokens))
        d.drf.copy_(adjusted.reshape(B * K, V))
        api.spec_adjust_logits(api.adjust_args(d.tgt, d.tgt, d.cu_q, max_q_rows=K + 1,
                                               draft_tokens=d.drafts, mask=dev(mask),
                                               mask_rows=dev(rows), **args))
        api.spec_verify_step(d.attn, d.sample, d.kv_cap, d.new_kv_len, d.ws)
        # 4. its tokens into the table
        api.spec_count_tokens(api.count_args(table.counts, table.seen, d.out_tokens, d.cu_q,
                                             num_accepted=d.num_accepted, slots=dev(slots),
                                             dev_status=status))
        torch.cuda.synchronize()
        want, _, _ = oracle.adjust_logits(inp["target_logits"], cu, draft_tokens=tokens, counts=ref,
                                          slots=slots, mask=mask, mask_rows=rows, **pen)
        _near(host_bits(d.tgt), want, slack)
        inp["target_logits"], inp["draft_logits"] = host_bits(d.tgt), host_bits(d.drf)
        inp["draft_tokens"] = tokens
        r = oracle.verify_step(inp)
        assert float(np.max(np.abs(d.out.float().cpu().numpy() - r["out"]))) < 2e-2
        acc, out = d.num_accepted.cpu().numpy(), d.out_tokens.cpu().numpy()
        n, ties = compare_sampling(r, acc, out, cu, tokens, V)
        if ties == 0:
            assert np.array_equal(d.new_kv_len.cpu().numpy(), r["new_kv_len"])
            assert np.array_equal(host_bits(d.k_cache), r["k_cache"])
            assert np.array_equal(host_bits(d.v_cache), r["v_cache"])
        ref, seen, _ = oracle.count_tokens(ref, out, cu, num_accepted=acc, slots=slots)
        assert np.array_equal(table.counts.cpu().numpy(), ref)
        assert np.array_equal(table.seen.cpu().numpy(), seen)
        assert int(status.item()) == 0 and d.status_bits() == 0
        # the next step starts from the device's caches and lengths
        inp["k_cache"], inp["v_cache"] = host_bits(d.k_cache), host_bits(d.v_cache)
        inp["kv_len"] = d.new_kv_len.cpu().numpy()


def test_a_step_captured_as_one_graph(api):
    """Rotary rows, adjustment, verify step and count in one graph, replayed on
    new inputs, against the same calls one by one."""
    inp = W.make_inputs(W.workload("bass_b8", B=4, V=3001, Hq=4, Hkv=4, L_lo=30, L_hi=200,
                                   gen_seed=61, cap_slack=20))
    turns, _ = api.rope_turns(128)

    def prepare():
        d = DeviceStep(inp, api)
        table = api.TokenCounts(4, 3001)
        rope = api.rope_args(d.q, d.k_new, None, d.q, d.k_new, None, turns, cu_q=d.cu_q,
                             kv_len=d.kv_len, max_q_rows=d.max_q_rows, dev_status=d.status)
        adjust = api.adjust_args(d.tgt, d.tgt, d.cu_q, max_q_rows=d.max_q_rows, draft=d.drf,
                                 draft_out=d.drf, draft_tokens=d.drafts, counts=table.counts,
                                 seen=table.seen, repetition=1.3, presence=0.4, frequency=0.3,
                                 dev_status=d.status)
        count = api.count_args(table.counts, table.seen, d.out_tokens, d.cu_q,
                               num_accepted=d.num_accepted, dev_status=d.status)

        def step():
            api.spec_rope_rows(rope)
            api.spec_adjust_logits(adjust)
            api.spec_verify_step(d.attn, d.sample, d.kv_cap, d.new_kv_len, d.ws)
            api.spec_count_tokens(count)
        return d, table, step

    (d1, t1, s1), (d2, t2, s2) = prepare(), prepare()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s1()
    for seed in range(3):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        for name in ("q", "k_new", "tgt", "drf"):
            x = getattr(d1, name)
            x.copy_(torch.randn(x.shape, generator=gen, device="cuda") * 2)
            getattr(d2, name).copy_(x)
        graph.replay()
        s2()
        torch.cuda.synchronize()
        for name in ("out", "num_accepted", "out_tokens", "new_kv_len", "k_cache", "v_cache", "tgt",
                     "drf"):
            assert torch.equal(getattr(d1, name), getattr(d2, name)), (seed, name)
        assert torch.equal(t1.counts, t2.counts) and torch.equal(t1.seen, t2.seen)
        assert int(t1.counts.sum()) > 0 and d1.status_bits() == d2.status_bits() == 0


def test_calls_in_the_shadow_of_other_kernels(api):
    """The operators' launches are worked on while the kernel before still runs: what
    it wrote has to be there, and what comes after has to see all of theirs, whether
    the neighbours are torch kernels, the attention, or each other."""
    inp = W.make_inputs(W.workload("bass_b8", B=4, V=40001, Hq=8, Hkv=8, L_lo=900, L_hi=2000,
                                   gen_seed=71, cap_slack=20))
    d = DeviceStep(inp, api)
    table = api.TokenCounts(4, 40001)
    turns, _ = api.rope_turns(128)
    x, y = torch.empty_like(d.q), torch.empty_like(d.q)
    logits, adjusted = torch.empty_like(d.tgt), torch.empty_like(d.tgt)
    tok = torch.zeros(4 * 700, dtype=torch.int32, device="cuda")
    start = torch.arange(5, dtype=torch.int32, device="cuda") * 700
    rope = api.rope_args(x, None, None, y, None, None, turns, cu_q=d.cu_q, kv_len=d.kv_len,
                         max_q_rows=d.max_q_rows)
    adjust = api.adjust_args(logits, adjusted, d.cu_q, max_q_rows=d.max_q_rows, counts=table.counts,
                             seen=table.seen, presence=1.0, frequency=0.5)
    reset = api.count_args(table.counts, table.seen, tok, start, reset=True)
    count = api.count_args(table.counts, table.seen, tok, start)
    big = torch.zeros(1 << 26, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(0)
    seen, want, turned = [], [], []
    for k in range(40):
        big.add_(1)                                     # a long kernel before
        tok.copy_(torch.randint(0, 40001, tok.shape, generator=gen, device="cuda"))
        api.spec_count_tokens(reset)
        api.spec_count_tokens(count)
        x.fill_(float(k + 1))
        api.spec_rope_rows(rope)
        api.spec_verify_attn(d.attn, d.ws)
        logits.fill_(float(k))
        api.spec_adjust_logits(adjust)
        seen.append(adjusted.clone())
        turned.append(y.clone())
        n = torch.zeros(4, 40001, device="cuda").scatter_add_(
            1, tok.view(4, 700).long(), torch.full((4, 700), 2.0, device="cuda"))
        less = torch.where(n > 0, 0.5 * n + 1.0, torch.zeros_like(n))
        want.append((float(k) - less).to(torch.bfloat16))
    torch.cuda.synchronize()
    rows = torch.repeat_interleave(torch.arange(4), torch.from_numpy(np.diff(inp["cu_q"])).long())
    for k in range(40):
        assert torch.equal(seen[k], want[k][rows.cuda()]), k
        # every pair (k + 1)(1, 1) turned keeps its length: sqrt(2) (k + 1), halves of steps apart
        pair = torch.hypot(turned[k][..., :64].float(), turned[k][..., 64:].float()) / (k + 1)
        assert float((pair - 2 ** 0.5).abs().max()) <= 2 ** 0.5 * 2.0 ** -8 + 1e-5, k


def test_inputs_written_by_the_kernel_just_before(api):
    """Each call reads what the launch before it on the stream has written (frequencies,
    tokens, logits), in buffers that the call before that one has read too."""
    n, V = 64, 5000
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(n, 2, 64, device="cuda", generator=g)
    pos = torch.arange(1, n + 1, device="cuda", dtype=torch.int64)
    tables = [api.rope_turns(64, base=b)[0] for b in (1e4, 1e6)]
    turns, y = torch.empty_like(tables[0]), torch.empty_like(x)
    rope = api.rope_args(x, None, None, y, None, None, turns, positions=pos)
    want = []
    for t in tables:
        turns.copy_(t)
        torch.cuda.synchronize()
        api.spec_rope_rows(rope)
        torch.cuda.synchronize()
        want.append(y.clone())
    assert not torch.equal(*want)
    prompts = torch.randint(0, V, (2, 4096), device="cuda", generator=g, dtype=torch.int32)
    start = torch.tensor([0, 4096], dtype=torch.int32, device="cuda")
    tokens, table = torch.empty_like(prompts[0]), api.TokenCounts(1, V)
    count = api.count_args(table.counts, table.seen, tokens, start, prompt=True, reset=True)
    marked = torch.zeros(2, V, dtype=torch.bool, device="cuda")
    for k in range(2):
        marked[k, prompts[k].long()] = True
    got_y, got_c = [], []
    for k in range(40):
        torch.mul(tables[k % 2], 1, out=turns)          # a kernel, not a copy
        api.spec_rope_rows(rope)
        got_y.append(y.clone())
        torch.add(prompts[k % 2], 0, out=tokens)
        api.spec_count_tokens(count)
        got_c.append(table.counts[0] < 0)
    torch.cuda.synchronize()
    for k in range(40):
        assert torch.equal(got_y[k], want[k % 2]), k
        assert torch.equal(got_c[k], marked[k % 2]), k


def test_captured_behind_copies_fills_and_another_stream(api):
    """In a graph, the operators may follow nodes that are no kernels (fills, copies) and
    join work of another stream: they wait for it all the same."""
    V, n = 4000, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(n, 2, 64, device="cuda", generator=g)
    xs, y, pos = torch.empty_like(x), torch.empty_like(x), torch.arange(n, device="cuda")
    turns, _ = api.rope_turns(64)
    rope = api.rope_args(xs, None, None, y, None, None, turns, positions=pos)
    logits = torch.randn(n, V, device="cuda", generator=g)
    ls, out = torch.empty_like(logits), torch.empty_like(logits)
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    tokens = torch.randint(0, V, (n,), device="cuda", generator=g, dtype=torch.int32)
    ts, table = torch.empty_like(tokens), api.TokenCounts(n, V)
    count = api.count_args(table.counts, table.seen, ts, cu)
    adjust = api.adjust_args(ls, out, cu, max_q_rows=1, counts=table.counts, seen=table.seen, presence=0.5)
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    main.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        table.counts.zero_()
        table.seen.zero_()
        ts.copy_(tokens)
        api.spec_count_tokens(count)                    # behind fills and a copy
        side.wait_stream(main)
        with torch.cuda.stream(side):
            ls.copy_(logits)
            xs.copy_(x)
            api.spec_rope_rows(rope)                    # behind a copy on the other stream
        main.wait_stream(side)
        api.spec_adjust_logits(adjust)                  # behind both streams
    for k in range(3):
        x.mul_(1.5)
        logits.mul_(-1.25)
        tokens.add_(7).remainder_(V)
        graph.replay()
        torch.cuda.synchronize()
        want = torch.empty_like(y)
        api.spec_rope_rows(api.rope_args(x, None, None, want, None, None, turns, positions=pos))
        assert torch.equal(y, want), k
        want = logits.clone()
        want[torch.arange(n, device="cuda"), tokens.long()] -= 0.5
        assert torch.equal(out, want), k
