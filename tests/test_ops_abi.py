"""The operators' C ABI (include/spec_ops.h): struct mirrors, refusals of bad
host arguments (nothing is launched, so no GPU is needed) and the checks of the
torch-facing calls."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def binding():
    from speculative_decoding_verify_09_gb300 import build
    build()
    from speculative_decoding_verify_09_gb300 import _binding
    return _binding


def test_struct_mirrors(binding):
    assert binding.lib.sv_ops_version() == 1
    for i, c in enumerate((binding.RopeArgs, binding.RopeScaling, binding.CountArgs,
                           binding.AdjustArgs)):
        assert binding.lib.sv_ops_struct_size(i) == ctypes.sizeof(c)
    assert binding.lib.sv_ops_struct_size(4) == 0


def _fill(a, kw):
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _rope(b, **kw):
    a = b.RopeArgs()
    a.batch, a.num_q_heads, a.num_kv_heads, a.head_dim, a.rot_dim = 2, 8, 2, 128, 64
    a.dtype, a.num_rows, a.max_q_rows = b.SV_BF16, 8, 5
    for k in ("turns", "cu_q", "kv_len", "q", "k", "v"):
        setattr(a, k, 4096)
    for k in ("q_out", "k_out", "v_out"):
        setattr(a, k, 1 << 20)
    return _fill(a, kw)


INVALID, UNSUPPORTED = 1, 4


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), INVALID), (dict(dtype=9), INVALID), (dict(kv_dtype=1), INVALID),
    (dict(num_q_heads=-1), INVALID), (dict(num_kv_heads=16385), INVALID), (dict(num_q_heads=16385), INVALID),
    (dict(head_dim=12), UNSUPPORTED), (dict(head_dim=0), UNSUPPORTED),
    (dict(head_dim=264, rot_dim=64), UNSUPPORTED),
    (dict(rot_dim=3), INVALID), (dict(rot_dim=0), INVALID), (dict(rot_dim=130), INVALID),
    (dict(layout=2), INVALID), (dict(layout=-1), INVALID),
    (dict(num_rows=-1), INVALID), (dict(num_rows=1 << 31), INVALID),
    (dict(mscale=-1.0), INVALID), (dict(mscale=float("nan")), INVALID),
    (dict(k_scale=float("inf")), INVALID), (dict(v_scale=-0.5), INVALID),
    (dict(batch=-1), INVALID), (dict(max_q_rows=0), INVALID),
    (dict(batch=1 << 20, max_q_rows=1 << 12), INVALID),
    (dict(cu_q=0), INVALID), (dict(kv_len=0), INVALID), (dict(turns=0), INVALID),
    (dict(q=0), INVALID), (dict(q_out=0), INVALID), (dict(k_out=0), INVALID),
    (dict(v_out=0), INVALID), (dict(q=4104), INVALID), (dict(k_out=4104), INVALID),
    (dict(q_stride=1016), INVALID), (dict(k_stride=257), INVALID), (dict(v_stride=-256), INVALID),
    (dict(q_stride=1028), INVALID), (dict(q_out=4096, q_stride=2048), INVALID),
    (dict(k_out=4096, kv_dtype=2), INVALID),
])
def test_rope_refusals(binding, kw, status):
    a = _rope(binding, **kw)
    assert binding.lib.spec_rope_rows(ctypes.byref(a), None) == status, binding.last_error()
    assert "rope" in binding.last_error()
    assert binding.lib.spec_rope_rows(None, None) == INVALID


@pytest.mark.parametrize("kw", [dict(num_rows=0), dict(num_rows=0, batch=0, cu_q=0, kv_len=0),
                                dict(num_rows=0, positions=4096, cu_q=0, kv_len=0),
                                dict(num_q_heads=0, k=0, v=0, q=0)])
def test_rope_with_nothing_to_do(binding, kw):
    a = _rope(binding, **kw)
    assert binding.lib.spec_rope_rows(ctypes.byref(a), None) == 0, binding.last_error()


def _count(b, **kw):
    a = b.CountArgs()
    a.batch, a.vocab, a.num_slots, a.num_tokens = 2, 1000, 4, 10
    for k in ("start", "tokens", "counts", "seen"):
        setattr(a, k, 4096)
    return _fill(a, kw)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), UNSUPPORTED), (dict(batch=65536), UNSUPPORTED), (dict(vocab=0), UNSUPPORTED),
    (dict(vocab=(1 << 23) + 1), UNSUPPORTED), (dict(num_slots=0), INVALID), (dict(flags=4), INVALID), (dict(num_tokens=-1), INVALID),
    (dict(num_tokens=1 << 31), INVALID), (dict(start=0), INVALID), (dict(tokens=0), INVALID),
    (dict(counts=0), INVALID), (dict(seen=0), INVALID),
])
def test_count_refusals(binding, kw, status):
    a = _count(binding, **kw)
    assert binding.lib.spec_count_tokens(ctypes.byref(a), None) == status, binding.last_error()
    assert "count" in binding.last_error()
    assert binding.lib.spec_count_tokens(None, None) == INVALID


def _adjust(b, **kw):
    a = b.AdjustArgs()
    a.batch, a.vocab, a.dtype, a.max_q_rows, a.num_rows = 2, 1000, b.SV_BF16, 5, 8
    a.num_slots, a.num_masks, a.num_bias, a.num_ctx = 4, 8, 3, 1
    for k in ("cu_q", "target", "draft", "draft_tokens", "counts", "seen", "bias_start",
              "bias_tokens", "bias_values", "mask", "ctx_tokens"):
        setattr(a, k, 4096)
    a.target_out = a.draft_out = 1 << 20
    return _fill(a, kw)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), UNSUPPORTED), (dict(batch=65536), UNSUPPORTED), (dict(vocab=0), UNSUPPORTED),
    (dict(vocab=(1 << 23) + 1), UNSUPPORTED),
    (dict(dtype=2), INVALID), (dict(max_q_rows=0), INVALID), (dict(max_q_rows=17), INVALID),
    (dict(num_rows=1), INVALID), (dict(num_rows=11), INVALID),
    (dict(repetition=-1.0), INVALID), (dict(repetition=float("inf")), INVALID),
    (dict(repetition=float("nan")), INVALID), (dict(repetition=1e-20), INVALID), (dict(presence=float("inf")), INVALID),
    (dict(frequency=float("nan")), INVALID), (dict(num_ctx=-1), INVALID),
    (dict(num_ctx=1025), INVALID), (dict(ctx_stride=-1), INVALID), (dict(ctx_tokens=0), INVALID),
    (dict(num_bias=-1), INVALID), (dict(num_bias=1 << 31), INVALID),
    (dict(bias_tokens=0), INVALID), (dict(bias_values=0), INVALID),
    (dict(num_slots=-1), INVALID), (dict(num_slots=0), INVALID), (dict(counts=0), INVALID),
    (dict(seen=0), INVALID), (dict(num_masks=-1), INVALID), (dict(num_masks=7), INVALID),
    (dict(mask_stride=31), INVALID), (dict(mask_stride=-32), INVALID),
    (dict(cu_q=0), INVALID), (dict(target=0), INVALID), (dict(target_out=0), INVALID),
    (dict(draft_out=0), INVALID), (dict(draft=0), INVALID),
    (dict(target=4104), INVALID), (dict(draft_out=(1 << 20) + 8), INVALID),
    (dict(target_out=4096), INVALID), (dict(draft_out=4096), INVALID),
])
def test_adjust_refusals(binding, kw, status):
    a = _adjust(binding, **kw)
    assert binding.lib.spec_adjust_logits(ctypes.byref(a), None) == status, binding.last_error()
    assert "adjust" in binding.last_error()
    assert binding.lib.spec_adjust_logits(None, None) == INVALID


def test_empty_batches_are_no_ops(binding):
    a, c = _adjust(binding, batch=0, num_rows=0), _count(binding, batch=0)
    assert binding.lib.spec_adjust_logits(ctypes.byref(a), None) == 0
    assert binding.lib.spec_count_tokens(ctypes.byref(c), None) == 0


def test_torch_calls_refuse_host_tensors(binding):
    import torch
    import speculative_decoding_verify_09_gb300 as pkg
    api = pkg.load()
    x = torch.zeros(2, 1, 64)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        api.rope_args(x, x, x, x, x, x, torch.zeros(32, dtype=torch.int64), cu_q=i, kv_len=i[:1],
                      max_q_rows=2)
    with pytest.raises(ValueError, match="CUDA"):
        api.adjust_args(x[:, 0], x[:, 0], i, max_q_rows=2)
    with pytest.raises(ValueError, match="CUDA"):
        api.count_args(torch.zeros(1, 8, dtype=torch.int32), i[:1].view(1, 1), i, i)


@pytest.mark.parametrize("std,compiler,lang", [("c99", "gcc", "c"), ("c++17", "g++", "c++")])
def test_header_compiles_as_plain_c_and_cxx(tmp_path, std, compiler, lang):
    src = tmp_path / "use_header.c"
    src.write_text('#include "spec_ops.h"\n'
                   "int main(void) {\n"
                   "  sv_rope_args r; sv_rope_scaling s; sv_count_args c; sv_adjust_args a;\n"
                   "  sv_status (*rope)(const sv_rope_args *, void *) = spec_rope_rows;\n"
                   "  sv_status (*adjust)(const sv_adjust_args *, void *) = spec_adjust_logits;\n"
                   "  sv_status (*count)(const sv_count_args *, void *) = spec_count_tokens;\n"
                   "  (void)r; (void)s; (void)c; (void)a; (void)rope; (void)adjust; (void)count;\n"
                   "  return 0;\n"
                   "}\n")
    r = subprocess.run([compiler, f"-std={std}", "-Wall", "-Wextra", "-Werror", "-pedantic",
                        "-x", lang, "-fsyntax-only", "-I", os.path.join(ROOT, "include"),
                        str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_as_many_tokens_or_biases_as_an_index_holds(binding):
    """The kernels step through both with a 32-bit index that must not wrap."""
    most = 1 << 30
    a = _count(binding, num_tokens=most + 1)
    assert binding.lib.spec_count_tokens(ctypes.byref(a), None) == INVALID
    assert "num_tokens" in binding.last_error()
    a = _adjust(binding, num_bias=most + 1)
    assert binding.lib.spec_adjust_logits(ctypes.byref(a), None) == INVALID
    assert "num_bias" in binding.last_error()
    # the largest that is allowed passes this check and meets the next one
    a = _count(binding, num_tokens=most, start=0)
    assert binding.lib.spec_count_tokens(ctypes.byref(a), None) == INVALID
    assert "start" in binding.last_error()
    a = _adjust(binding, num_bias=most, num_slots=-1)
    assert binding.lib.spec_adjust_logits(ctypes.byref(a), None) == INVALID
    assert "num_slots" in binding.last_error()


def test_kernels_launched_behind_another_read_by_ordinary_loads():
    """They may be resident while the kernel before them still writes what they
    read: the read-only path is not for them."""
    csrc = os.path.join(ROOT, "speculative_decoding_verify_09_gb300", "csrc")
    found = 0
    for name in sorted(os.listdir(csrc)):
        with open(os.path.join(csrc, name)) as fh:
            code = "\n".join(ln.split("//")[0] for ln in fh)
        if "launch_behind(" in code and name.endswith(".cu"):
            found += 1
            assert "__ldg" not in code and "ld.global.nc" not in code, name
    assert found == 2
