"""The C ABI of the norms and the 4-bit cache (include/spec_kv4.h): struct
mirrors, refusals of bad host arguments (nothing is launched, so no GPU is
needed), the checks of the torch-facing calls, and the loads of the kernels."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, WORKSPACE, UNSUPPORTED = 1, 2, 4


@pytest.fixture(scope="module")
def binding():
    from speculative_decoding_verify_09_gb300 import build
    build()
    from speculative_decoding_verify_09_gb300 import _binding
    return _binding


def test_struct_mirrors(binding):
    assert binding.lib.sv_kv4_version() == 1
    for i, c in enumerate((binding.Kv4Cache, binding.NormArgs, binding.NormRopeArgs,
                           binding.Kv4AppendArgs, binding.Kv4ReadArgs, binding.Kv4AttnArgs)):
        assert binding.lib.sv_kv4_struct_size(i) == ctypes.sizeof(c)
    assert binding.lib.sv_kv4_struct_size(6) == 0


def _set(a, kw):
    """Fields by dotted name."""
    for k, v in kw.items():
        *path, last = k.split("__")
        x = a
        for p in path:
            x = getattr(x, p)
        assert hasattr(x, last), k
        setattr(x, last, v)
    return a


def _rows(b, a):
    a.batch, a.num_q_heads, a.num_kv_heads, a.head_dim, a.rot_dim = 2, 8, 2, 128, 64
    a.dtype, a.num_rows, a.max_q_rows = b.SV_BF16, 8, 5
    for k in ("turns", "cu_q", "kv_len", "q", "k", "v"):
        setattr(a, k, 4096)
    for k in ("q_out", "k_out", "v_out"):
        setattr(a, k, 1 << 20)


def _cache(a):
    a.num_kv_heads, a.head_dim, a.page_size, a.max_pages, a.num_pages = 2, 128, 64, 4, 10
    a.pages, a.table = 1 << 21, 4096


def _norm_rope(b, **kw):
    a = b.NormRopeArgs()
    _rows(b, a.rope)
    a.norm.eps = 1e-6
    a.norm.q_weight = a.norm.k_weight = 4096
    return _set(a, kw)


def _append(b, **kw):
    a = b.Kv4AppendArgs()
    _rows(b, a.rows)
    a.rows.k_out = a.rows.v_out = 0
    _cache(a.cache)
    return _set(a, kw)


def _read(b, **kw):
    a = b.Kv4ReadArgs()
    _cache(a.cache)
    a.batch, a.max_q_rows, a.dtype, a.num_rows = 2, 5, b.SV_BF16, 8
    a.cu_q = a.kv_len = 4096
    a.k_out = a.v_out = 1 << 20
    return _set(a, kw)


def _attn(b, **kw):
    a = b.Kv4AttnArgs()
    _cache(a.cache)
    a.batch, a.num_q_heads, a.max_q_rows, a.dtype, a.num_rows = 2, 8, 5, b.SV_BF16, 8
    a.cu_q = a.kv_len = a.q = 4096
    a.out = 1 << 20
    return _set(a, kw)


NAN, INF = float("nan"), float("inf")
BAD_CACHE = [
    (dict(cache__head_dim=96), UNSUPPORTED), (dict(cache__head_dim=0), UNSUPPORTED),
    (dict(cache__num_kv_heads=0), INVALID), (dict(cache__num_kv_heads=1025), INVALID),
    (dict(cache__page_size=0), INVALID), (dict(cache__page_size=24), INVALID),
    (dict(cache__page_size=4112), INVALID), (dict(cache__max_pages=-1), INVALID),
    (dict(cache__table_stride=3), INVALID), (dict(cache__table_stride=-4), INVALID),
    (dict(cache__num_pages=0), INVALID), (dict(cache__num_pages=1 << 31), INVALID),
    (dict(cache__k_scale=-1.0), INVALID), (dict(cache__v_scale=NAN), INVALID),
    (dict(cache__k_scale=INF), INVALID), (dict(cache__v_scale=1e-30), INVALID),
    (dict(cache__pages=0), INVALID), (dict(cache__pages=(1 << 21) + 8), INVALID),
    (dict(cache__table=0), INVALID),
]


@pytest.mark.parametrize("kw,status", [
    (dict(rope__dtype=2), INVALID), (dict(rope__kv_dtype=1), INVALID),
    (dict(rope__num_q_heads=-1), INVALID), (dict(rope__head_dim=12), UNSUPPORTED),
    (dict(rope__head_dim=264, rope__rot_dim=64), UNSUPPORTED), (dict(rope__rot_dim=3), INVALID),
    (dict(rope__rot_dim=130), INVALID), (dict(rope__layout=2), INVALID),
    (dict(rope__num_rows=-1), INVALID), (dict(rope__mscale=NAN), INVALID),
    (dict(rope__batch=-1), INVALID), (dict(rope__max_q_rows=0), INVALID),
    (dict(rope__cu_q=0), INVALID), (dict(rope__q=0), INVALID), (dict(rope__k_out=0), INVALID),
    (dict(rope__q=4104), INVALID), (dict(rope__q_stride=1028), INVALID),
    (dict(rope__turns=0, rope__kv_len=0), INVALID), (dict(rope__q_out=4096, rope__q_stride=2048), INVALID),
    (dict(norm__eps=-1e-6), INVALID), (dict(norm__eps=NAN), INVALID), (dict(norm__eps=INF), INVALID),
    (dict(norm__weight_offset=INF), INVALID), (dict(norm__q_weight=4098), INVALID),
    (dict(norm__k_weight=4097), INVALID),
])
def test_norm_rope_refusals(binding, kw, status):
    a = _norm_rope(binding, **kw)
    assert binding.lib.spec_norm_rope_rows(ctypes.byref(a), None) == status, binding.last_error()
    assert binding.last_error().startswith("norm_rope: ")
    assert binding.lib.spec_norm_rope_rows(None, None) == INVALID


@pytest.mark.parametrize("kw,status", BAD_CACHE + [
    (dict(rows__positions=4096), INVALID), (dict(rows__num_kv_heads=4), INVALID),
    (dict(rows__head_dim=64), INVALID), (dict(rows__k=0), INVALID), (dict(rows__v=0), INVALID),
    (dict(rows__q_out=0), INVALID), (dict(rows__q=0), INVALID), (dict(rows__dtype=2), INVALID),
    (dict(rows__k=1 << 21), INVALID), (dict(rows__v=1 << 21), INVALID), (dict(rows__k=4104), INVALID),
    (dict(rows__v_stride=255), INVALID), (dict(rows__rot_dim=130), INVALID),
    (dict(rows__layout=-1), INVALID), (dict(rows__max_q_rows=0), INVALID),
    (dict(rows__batch=-1), INVALID), (dict(rows__kv_len=0), INVALID),
    (dict(rows__batch=1 << 20, rows__max_q_rows=1 << 12), INVALID), (dict(norm__eps=-1.0), INVALID),
    (dict(norm__k_weight=4097), INVALID),
])
def test_append_refusals(binding, kw, status):
    a = _append(binding, **kw)
    assert binding.lib.spec_kv4_append(ctypes.byref(a), None) == status, binding.last_error()
    assert binding.last_error().startswith("kv4_append: ")
    assert binding.lib.spec_kv4_append(None, None) == INVALID


@pytest.mark.parametrize("kw,status", BAD_CACHE + [
    (dict(batch=-1), INVALID), (dict(max_q_rows=0), INVALID),
    (dict(batch=1 << 20, max_q_rows=1 << 12), INVALID), (dict(dtype=7), INVALID),
    (dict(reserved=1), INVALID), (dict(num_rows=-1), INVALID), (dict(num_rows=1 << 31), INVALID),
    (dict(k_out_scale=-1.0), INVALID), (dict(v_out_scale=INF), INVALID), (dict(cu_q=0), INVALID),
    (dict(kv_len=0), INVALID), (dict(k_out=(1 << 20) + 8), INVALID), (dict(v_out=4104), INVALID),
])
def test_read_refusals(binding, kw, status):
    a = _read(binding, **kw)
    assert binding.lib.spec_kv4_read(ctypes.byref(a), None) == status, binding.last_error()
    assert binding.last_error().startswith("kv4_read: ")
    assert binding.lib.spec_kv4_read(None, None) == INVALID


BAD_SHAPES = [
    (dict(batch=-1), UNSUPPORTED), (dict(batch=769), UNSUPPORTED), (dict(num_q_heads=0), INVALID),
    (dict(num_q_heads=7), INVALID), (dict(num_q_heads=1026), INVALID), (dict(dtype=0), UNSUPPORTED),
    (dict(dtype=2), UNSUPPORTED), (dict(reserved=1), INVALID), (dict(max_q_rows=0), INVALID),
    (dict(max_q_rows=1025), INVALID), (dict(num_rows=-1), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID), (dict(q_stride=1023), INVALID),
    (dict(q_stride=1028), INVALID), (dict(q_stride=-1024), INVALID),
    (dict(batch=768, cache__num_kv_heads=128, num_q_heads=128), UNSUPPORTED),
    (dict(max_q_rows=1024, num_q_heads=512), UNSUPPORTED),
    (dict(cache__max_pages=1 << 27), UNSUPPORTED),
    (dict(batch=768, cache__max_pages=1 << 20), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", BAD_CACHE + BAD_SHAPES + [
    (dict(cu_q=0), INVALID), (dict(kv_len=0), INVALID), (dict(q=0), INVALID), (dict(out=0), INVALID),
    (dict(q=4104), INVALID), (dict(out=(1 << 20) + 8), INVALID), (dict(out=4096), INVALID),
])
def test_attn_refusals(binding, kw, status):
    a = _attn(binding, **kw)
    ws = ctypes.c_void_p(4096)
    assert binding.lib.spec_kv4_attn(ctypes.byref(a), ws, 1 << 30, None) == status, binding.last_error()
    assert binding.last_error().startswith("kv4_attn: ")
    if (kw, status) in BAD_SHAPES:
        assert binding.lib.sv_kv4_workspace_bytes(ctypes.byref(a)) == 0
    assert binding.lib.spec_kv4_attn(None, ws, 1 << 30, None) == INVALID
    assert binding.lib.sv_kv4_workspace_bytes(None) == 0


def test_attn_workspace(binding):
    a = _attn(binding)
    need = binding.lib.sv_kv4_workspace_bytes(ctypes.byref(a))
    assert need > 0 and need % 256 == 0
    for ws, n in ((0, need), (4096, need - 1), (4096 + 128, need)):
        assert binding.lib.spec_kv4_attn(ctypes.byref(a), ctypes.c_void_p(ws), n, None) == WORKSPACE
    # the size is known before any tensor is
    b = _attn(binding, cu_q=0, kv_len=0, q=0, out=0, cache__pages=0, cache__table=0)
    assert binding.lib.sv_kv4_workspace_bytes(ctypes.byref(b)) == need


def test_nothing_to_do(binding):
    for kw in (dict(rope__num_rows=0), dict(rope__num_rows=0, rope__batch=0, rope__cu_q=0, rope__kv_len=0),
               dict(rope__num_rows=0, rope__turns=0)):
        a = _norm_rope(binding, **kw)
        assert binding.lib.spec_norm_rope_rows(ctypes.byref(a), None) == 0, binding.last_error()
    a = _append(binding, rows__num_rows=0, rows__k=0, rows__v=0, rows__q=0)
    assert binding.lib.spec_kv4_append(ctypes.byref(a), None) == 0, binding.last_error()
    for kw in (dict(num_rows=0), dict(batch=0, cu_q=0, kv_len=0), dict(k_out=0, v_out=0)):
        a = _read(binding, **kw)
        assert binding.lib.spec_kv4_read(ctypes.byref(a), None) == 0, binding.last_error()
    for kw in (dict(num_rows=0, q=0, out=0), dict(batch=0, cu_q=0, kv_len=0)):
        a = _attn(binding, **kw)
        assert binding.lib.spec_kv4_attn(ctypes.byref(a), ctypes.c_void_p(4096), 1 << 30, None) == 0


def test_torch_calls_refuse(binding):
    import torch
    import speculative_decoding_verify_09_gb300 as pkg
    api = pkg.load()
    x, i = torch.zeros(2, 1, 64), torch.zeros(2, dtype=torch.int32)
    t = torch.zeros(1, 1, dtype=torch.int32)
    cache = api.Kv4Cache(1, 1, 64, device="cpu")
    assert cache.pages.shape == (1, 1, 4, 18 * 64)
    with pytest.raises(ValueError, match="CUDA"):
        api.norm_rope_args(x, x, x, x, x, x, cu_q=i, kv_len=i[:1], max_q_rows=2)
    with pytest.raises(ValueError, match="CUDA"):
        api.kv4_append_args(cache, t, i, i[:1], x, x, max_q_rows=2)
    with pytest.raises(ValueError, match="CUDA"):
        api.kv4_read_args(cache, t, i, i[:1], x, x, max_q_rows=2)
    with pytest.raises(ValueError, match="CUDA"):
        api.kv4_attn_args(cache, t, i, i[:1], x, x, max_q_rows=2)
    with pytest.raises(ValueError, match="both None"):
        api.kv4_read_args(cache, t, i, i[:1], None, None, max_q_rows=2)
    with pytest.raises(ValueError, match="needed"):
        api.kv4_append_args(cache, t, i, i[:1], x, None, max_q_rows=2)
    with pytest.raises(ValueError, match="page_size"):
        api.Kv4Cache(1, 1, 64, page_size=40, device="cpu")
    with pytest.raises(ValueError, match="pages"):
        api.Kv4Cache(1, 1, 64, pages=torch.zeros(1, 1, 4, 100, dtype=torch.uint8))


@pytest.mark.parametrize("std,compiler,lang", [("c99", "gcc", "c"), ("c++17", "g++", "c++")])
def test_header_compiles_as_plain_c_and_cxx(tmp_path, std, compiler, lang):
    src = tmp_path / "use_header.c"
    src.write_text('#include "spec_kv4.h"\n'
                   "int main(void) {\n"
                   "  sv_norm_rope_args n; sv_kv4_append_args p; sv_kv4_read_args r; sv_kv4_attn_args a;\n"
                   "  sv_status (*norm)(const sv_norm_rope_args *, void *) = spec_norm_rope_rows;\n"
                   "  sv_status (*append)(const sv_kv4_append_args *, void *) = spec_kv4_append;\n"
                   "  sv_status (*read)(const sv_kv4_read_args *, void *) = spec_kv4_read;\n"
                   "  sv_status (*attn)(const sv_kv4_attn_args *, void *, size_t, void *) = spec_kv4_attn;\n"
                   "  (void)n; (void)p; (void)r; (void)a; (void)norm; (void)append; (void)read; (void)attn;\n"
                   "  return 0;\n"
                   "}\n")
    r = subprocess.run([compiler, f"-std={std}", "-Wall", "-Wextra", "-Werror", "-pedantic",
                        "-x", lang, "-fsyntax-only", "-I", os.path.join(ROOT, "include"),
                        str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_kernels_launched_behind_another_read_by_ordinary_loads():
    """They may be resident while the kernel before them still writes what they
    read: the read-only path is not for them, nor for what they include."""
    csrc = os.path.join(ROOT, "speculative_decoding_verify_09_gb300", "csrc")
    found = []
    for name in sorted(os.listdir(csrc)):
        with open(os.path.join(csrc, name)) as fh:
            code = "\n".join(ln.split("//")[0] for ln in fh)
        if ("launch_after_previous(" in code and name.endswith(".cu")) or name.endswith(".inl"):
            found.append(name)
            assert "__ldg" not in code and "ld.global.nc" not in code, name
    assert {"norm_rope.cu", "kv4_attn.cu", "kv4.inl", "rows.inl"} <= set(found)
