"""Host side of the paged cache: the C ABI's argument checks, the binding's
metadata checks (CPU tensors; a valid call stops at the device check), and pins
of the float64 oracle that the GPU tests compare with."""
import ctypes
import os
import subprocess
import sys
import warnings

import numpy as np
import pytest
import torch

import oracle
from learnable_sink_b200 import sinkattn as S

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
bf, f16, f32, i32 = torch.bfloat16, torch.float16, torch.float32, torch.int32
B, Hq, Hkv, D, PAGE, NP, MP = 3, 8, 2, 64, 16, 12, 4


# ------------------------------------------------------------------ C ABI
def _struct(**kw):
    a = 256  # stand-in 16-byte-aligned device address: never dereferenced here
    c = S.CPagedCache(a, a, None, None, a, a, B, NP, PAGE, MP, Hkv, D)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _append(dt=0, T=B, Hq=Hq, c=None, k=256, ks=Hkv * D, v=256, vs=Hkv * D, q=None, qs=0, cu=None,
            rope=None, rot=0, n_pos=0, il=0, q_out=None, k_out=None, fp8=False):
    c = _struct() if c is None else c
    f = S.lib().sinkattn_paged_append_fp8 if fp8 else S.lib().sinkattn_paged_append
    return f(dt, T, Hq, ctypes.byref(c), k, ks, v, vs, q, qs, cu, rope, rot, n_pos, il, q_out,
             k_out, None)


def _decode(dt=0, Hq=Hq, q=256, c=None, n_sink=0, window=0, out=256, lse=256, ws=256,
            nb=1 << 24, fp8=False):
    c = _struct() if c is None else c
    f = S.lib().sinkattn_paged_decode_fp8 if fp8 else S.lib().sinkattn_paged_decode
    return f(dt, Hq, 0.1, q, ctypes.byref(c), n_sink, window, None, out, lse, None, ws, nb, None)


CALLS = {"append": _append, "decode": _decode}


@pytest.mark.parametrize("call", sorted(CALLS))
@pytest.mark.parametrize("field,value,code", [
    ("B", 0, 1), ("B", 65536, 1), ("n_pages", 0, 1), ("max_pages", 0, 1), ("Hkv", 0, 1),
    ("Hkv", 3, 1), ("D", 96, 1), ("page_size", 24, 2), ("page_size", 8, 2), ("page_size", 256, 2),
    ("page_size", 0, 2), ("k_pages", None, 1), ("v_pages", 264, 1), ("block_table", None, 1),
    ("cache_seqlens", None, 1), ("k_scale", 256, 1), ("n_pages", 1 << 27, 1),
    ("max_pages", 1 << 28, 1)])
def test_cache_descriptor_is_checked(call, field, value, code):
    kw = {}
    if field == "B" and call == "append" and value > 0:
        kw["T"] = value
    assert CALLS[call](c=_struct(**{field: value}), **kw) == code


def test_append_arguments_are_checked():
    assert _append(dt=2) == 2                       # float32
    assert _append(dt=7) == 1
    assert _append(T=-1) == 1
    assert _append(T=B + 1) == 1                    # one token a sequence without cu_new
    assert _append(k=None) == 1
    assert _append(v=264) == 1
    assert _append(ks=Hkv * D - 8) == 1             # overlapping tokens
    assert _append(ks=Hkv * D + 4) == 1             # tokens not 16-byte aligned
    assert _append(q=256, qs=Hq * D) == 1           # no q_out
    assert _append(q_out=256) == 1                  # no q
    assert _append(q=256, qs=Hkv * D, q_out=256) == 1
    assert _append(k_out=264) == 1
    for rot in (0, 8, 24, 80):
        assert _append(rope=256, rot=rot, n_pos=9) == 1
    assert _append(rope=256, rot=32, n_pos=0) == 1
    assert _append(il=2) == 1
    assert _append(fp8=True) == 1                   # no scales
    ok8 = _struct(k_scale=256, v_scale=256)
    assert _append(c=ok8) == 1                      # scales with the 16-bit call
    assert _append(c=_struct(k_scale=256), fp8=True) == 1


def test_decode_arguments_are_checked():
    assert _decode(dt=2) == 2
    assert _decode(q=None) == 1
    assert _decode(out=264) == 1
    assert _decode(lse=None) == 1
    assert _decode(ws=None) == 1
    assert _decode(n_sink=-1) == 1
    assert _decode(window=-1) == 1
    assert _decode(Hq=7) == 1
    assert _decode(fp8=True) == 1
    assert _decode(c=_struct(k_scale=256, v_scale=256)) == 1
    if torch.cuda.is_available():
        assert _decode(Hq=34) == 2                  # 17 query heads a KV head
        assert _decode(nb=16) == 4


def test_workspace_query():
    f = S.paged_decode_workspace_bytes
    assert f(0, 8, 2, 64) == 0 and f(1, 7, 2, 64) == 0 and f(1, 8, 2, 96) == 0
    # a partial of every query head for each sequence and KV head at least
    assert f(32, 32, 8, 128) >= 32 * 32 * 130 * 4


def test_decode_schedule_covers_every_position_once(tmp_path):
    """The paged decode's schedule (host code, compiled and run on the CPU): every
    visible position in one tile, partial slots distinct and inside the workspace."""
    from learnable_sink_b200 import build
    exe = str(tmp_path / "paged_schedule_check")
    subprocess.check_call([build.nvcc(), "-std=c++17", "-arch=sm_100a", "-I", os.path.join(ROOT, "include"),
                           os.path.join(ROOT, "tests", "c", "paged_schedule_check.cu"), "-o", exe])
    out = subprocess.run([exe], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.startswith("ok "), out.stdout


def test_decode_schedule_of_groups(tmp_path):
    """The schedule as the kernels use it, by the functions that they call: groups of CTAs, rows
    cut and rows left whole, partial slots, and the join's own reckoning of the segments."""
    from learnable_sink_b200 import build
    exe = str(tmp_path / "paged_groups_check")
    subprocess.check_call([build.nvcc(), "-O2", "-std=c++17", "-arch=sm_100a", "--expt-relaxed-constexpr",
                           "-I", os.path.join(ROOT, "include"),
                           os.path.join(ROOT, "tests", "c", "paged_groups_check.cu"), "-o", exe])
    out = subprocess.run([exe], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.startswith("ok "), out.stdout


# ------------------------------------------------------------------ binding
def _pool(dtype=bf, n=NP, h=Hkv, page=PAGE, d=D):
    return torch.zeros(n, h, page, d, dtype=dtype)


def _table(b=B, dtype=i32):
    return torch.zeros(b, MP, dtype=dtype)


def _refused(call, what):
    with pytest.raises(S.SinkAttnError, match=what) as e:
        call()
    assert e.value.code == 1


def test_cache_constructor_checks():
    lens = torch.zeros(B, dtype=i32)
    sc = torch.ones(NP, Hkv)
    C = S.PagedCache
    for ok in (lambda: C(_pool(), _pool(), _table(), lens),
               lambda: C(_pool(f16), _pool(f16), _table(), lens),
               lambda: C(_pool(torch.uint8), _pool(torch.uint8), _table(), lens, sc, sc),
               lambda: C(_pool(torch.float8_e4m3fn), _pool(torch.float8_e4m3fn), _table(), lens, sc, sc)):
        with pytest.raises(ValueError, match="contiguous CUDA tensors"):
            ok()
    _refused(lambda: C(_pool()[0], _pool(), _table(), lens), "pages must be")
    _refused(lambda: C(_pool(), _pool(f16), _table(), lens), "v_pages")
    _refused(lambda: C(_pool(), _pool(n=NP + 1), _table(), lens), "v_pages")
    _refused(lambda: C(_pool(f32), _pool(f32), _table(), lens), "pages are")
    _refused(lambda: C(_pool(torch.float8_e5m2), _pool(torch.float8_e5m2), _table(), lens, sc, sc),
             "pages are")
    _refused(lambda: C(_pool(torch.uint8), _pool(torch.uint8), _table(), lens), "need scales")
    _refused(lambda: C(_pool(torch.uint8), _pool(torch.uint8), _table(), lens, sc, sc[:, :1]),
             "v_scale")
    _refused(lambda: C(_pool(torch.uint8), _pool(torch.uint8), _table(), lens, sc.half(), sc),
             "k_scale")
    _refused(lambda: C(_pool(), _pool(), _table(), lens, sc, sc), "scales go with")
    _refused(lambda: C(_pool(page=24), _pool(page=24), _table(), lens), "page_size 24")
    _refused(lambda: C(_pool(d=96), _pool(d=96), _table(), lens), "D 96")
    _refused(lambda: C(_pool(), _pool(), _table(dtype=torch.int64), lens), "block_table")
    _refused(lambda: C(_pool(), _pool(), _table(), lens.long()), "cache_seqlens")
    _refused(lambda: C(_pool(), _pool(), _table(), lens[:2]), "cache_seqlens")


@pytest.fixture
def caches(monkeypatch):
    """A 16-bit and an 8-bit cache of CPU tensors (their device check skipped)."""
    with monkeypatch.context() as m:
        m.setattr(S, "_contig", lambda *a: None)
        lens = torch.zeros(B, dtype=i32)
        sc = torch.ones(NP, Hkv)
        return (S.PagedCache(_pool(), _pool(), _table(), lens),
                S.PagedCache(_pool(torch.uint8), _pool(torch.uint8), _table(), lens, sc, sc))


def test_cache_attributes_are_fixed(caches):
    """The calls use the addresses that the constructor checked: putting another tensor
    in an attribute is refused, not ignored."""
    for c in caches:
        for name in ("cache_seqlens", "block_table", "k_pages", "k_scale", "B", "_kind"):
            with pytest.raises(AttributeError, match=name):
                setattr(c, name, torch.ones(B, dtype=i32))
        assert c.cache_seqlens.tolist() == [0] * B


def test_cache_attributes_stay(caches):
    """Deleting an attribute would free memory that the descriptor names."""
    for c in caches:
        for name in ("k_pages", "block_table", "cache_seqlens", "_c", "_kind"):
            with pytest.raises(AttributeError, match=name):
                delattr(c, name)
        assert c.k_pages.shape[0] == NP and c.cache_seqlens.tolist() == [0] * B


def test_append_metadata_mismatches_are_refused(caches):
    c16, c8 = caches
    T = 7
    k = torch.zeros(T, Hkv, D, dtype=bf)
    q = torch.zeros(T, Hq, D, dtype=bf)
    cu = torch.tensor([0, 2, 2, 7], dtype=i32)
    rope = torch.zeros(9, 32)
    A = S.paged_append
    _refused(lambda: A(k.half(), k.half(), c16, cu), "k is")
    _refused(lambda: A(k, k, c8, cu), "k is")
    _refused(lambda: S.paged_append_fp8(k, k, c16, cu), "not an 8-bit cache")
    _refused(lambda: A(k, k.half(), c16, cu), "v is")
    _refused(lambda: A(k, k[:5], c16, cu), "v has shape")
    _refused(lambda: A(k[:, :1], k[:, :1], c16, cu), "k has shape")
    _refused(lambda: A(k, k, c16), "7 tokens for 3 sequences")
    _refused(lambda: A(k, k, c16, cu.long()), "cu_new")
    _refused(lambda: A(k, k, c16, cu[:3]), "cu_new")
    _refused(lambda: A(k.transpose(1, 2).contiguous().transpose(1, 2), k, c16, cu), "contiguous")
    _refused(lambda: A(torch.zeros(T, Hkv + 1, D, dtype=bf)[:, :, :].view(-1)[4:4 + T * Hkv * D]
                       .view(T, Hkv, D), k, c16, cu), "16-byte aligned")
    _refused(lambda: A(k[:1].expand(T, Hkv, D), k, c16, cu), "overlap")
    _refused(lambda: A(k, k, c16, cu, q_out=q), "q_out without q")
    _refused(lambda: A(k, k, c16, cu, q=q, q_out=q[:, :4]), "q_out")
    _refused(lambda: A(k, k, c16, cu, q=q, q_out=q.float()), "q_out")
    _refused(lambda: A(k, k, c16, cu, k_out=k[:5]), "k_out")
    _refused(lambda: A(k, k, c16, cu, rope=rope.double()), "rope")
    _refused(lambda: A(k, k, c16, cu, rope=rope[:, ::2]), "rope")
    _refused(lambda: A(k, k, c16, cu, rope=torch.zeros(9, 24)), "rot_dim 24")
    _refused(lambda: A(k, k, c16, cu, rope=torch.zeros(9, 128)), "rot_dim 128")


def test_decode_metadata_mismatches_are_refused(caches):
    c16, c8 = caches
    q = torch.zeros(B, Hq, D, dtype=bf)
    sink = torch.zeros(Hq)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    _refused(lambda: S.paged_decode(q[:2], c16, sink, workspace=ws), "disagree on B or D")
    _refused(lambda: S.paged_decode(q.half(), c16, sink, workspace=ws), "k_pages")
    _refused(lambda: S.paged_decode(q, c8, sink, workspace=ws), "k_pages")
    _refused(lambda: S.paged_decode_fp8(q, c16, sink, workspace=ws), "not an 8-bit cache")
    _refused(lambda: S.paged_decode(q, c16, sink[:4], workspace=ws), "learnable_sink")
    _refused(lambda: S.paged_decode(q, c16, sink, workspace=ws, out=q.float()), "out")
    _refused(lambda: S.paged_decode(q, c16, sink, workspace=ws, lse=torch.zeros(B, 1)), "lse")
    _refused(lambda: S.paged_decode(q, c16, sink, workspace=ws, sink_s=torch.zeros(B, 1)), "sink_s")


def test_decode_window_and_sink_tokens_out_of_range_are_refused(caches):
    """Not cut to their low 32 bits (2^32 + 5 would see five positions)."""
    q, z = torch.zeros(B, Hq, D, dtype=bf), torch.zeros(B, Hq)
    for kw in (dict(window=2 ** 32 + 5), dict(n_sink=2 ** 32), dict(window=2 ** 31), dict(window=4.5),
               dict(n_sink=-1), dict(window=-2 ** 32 + 7)):
        for c, call in zip(caches, (S.paged_decode, S.paged_decode_fp8)):
            _refused(lambda: call(q, c, None, workspace=z, out=q, lse=z, sink_s=z, **kw), "whole number")


def test_short_way_declines_what_it_does_not_handle(caches):
    """The extension makes no call for tensors off the GPU, other objects, or values
    out of range: the Python path then says what is wrong."""
    c16, _ = caches
    k = torch.zeros(B, Hkv, D, dtype=bf)
    a = S._short_way().paged_append
    head = (c16._at, 0, c16._kind, c16._dev)
    assert a(*head, k, k, None, None, False, None, None, None) == -1
    assert a(*head, "k", k, None, None, False, None, None, None) == -1
    assert a(0, 0, 0, 0, k, k, None, None, False, None, None, None) == -1
    d = S._short_way().paged_decode
    q = torch.zeros(B, Hq, D, dtype=bf)
    assert d(*head, q, None, 0, 0, None, q, q, q, q) == -1
    with pytest.raises(TypeError):
        d(1, 2)


@pytest.mark.parametrize("broken", ["missing", "other torch"])
def test_without_the_extension_the_python_path_makes_the_calls(caches, monkeypatch, broken):
    """A missing _binding.so, or one of another torch, is said once and does not stop the calls."""
    import learnable_sink_b200 as pkg
    if broken == "missing":
        monkeypatch.delattr(pkg, "_binding", raising=False)
        monkeypatch.setitem(sys.modules, "learnable_sink_b200._binding", None)
    else:
        monkeypatch.setattr(torch, "__version__", "1.0.0+cpu")
    monkeypatch.setattr(S, "_short", None)
    c16, c8 = caches
    k = torch.zeros(B, Hkv, D, dtype=bf)
    q, z = torch.zeros(B, Hq, D, dtype=bf), torch.zeros(B, Hq)
    with pytest.warns(RuntimeWarning, match="_binding.so"):
        _refused(lambda: S.paged_append(k.half(), k.half(), c16), "k is")
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        _refused(lambda: S.paged_decode_fp8(q, c16, None, workspace=z, out=q, lse=z, sink_s=z),
                 "not an 8-bit cache")


def test_build_makes_the_library_before_the_extension(monkeypatch):
    """Without g++ or torch's headers the library is built all the same, and the failure said."""
    from learnable_sink_b200 import build
    order = []
    compile_ = build._compile

    def no_extension(*a):
        order.append("extension")
        raise RuntimeError("g++ failed")

    monkeypatch.setattr(build, "_compile", lambda *a: order.append("library") or compile_(*a))
    monkeypatch.setattr(build, "build_binding", no_extension)
    with pytest.raises(RuntimeError, match="g[+][+] failed"):
        build.build()
    assert order[0] == "library" and order[-1] == "extension" and order.count("extension") == 1
    assert os.path.exists(build.LIB)


def test_build_compiles_the_extension_again_for_another_torch(monkeypatch):
    from learnable_sink_b200 import build
    build.build_binding()
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        return subprocess.CompletedProcess(cmd, 1, "", "")

    monkeypatch.setattr(build.subprocess, "run", run)
    build.build_binding()
    assert not ran
    monkeypatch.setattr(torch, "__version__", "1.0.0")
    with pytest.raises(RuntimeError, match="binding"):
        build.build_binding()
    assert len(ran) == 1 and "binding.cpp" in " ".join(ran[0])


# ------------------------------------------------------------------ the oracle
def test_oracle_rotation_closed_forms():
    rope = oracle.rope_table(40, 4, base=100.0)
    # angles p and p / 10
    assert np.allclose(rope[7], [np.cos(7), np.cos(0.7), np.sin(7), np.sin(0.7)])
    x = np.zeros((1, 1, 6))
    x[0, 0] = [1, 2, 3, 4, 5, 6]
    y = oracle.rotate(x, [7], rope)[0, 0]
    assert np.allclose(y[[0, 2]], [np.cos(7) - 3 * np.sin(7), 3 * np.cos(7) + np.sin(7)])
    assert np.allclose(y[[1, 3]], [2 * np.cos(.7) - 4 * np.sin(.7), 4 * np.cos(.7) + 2 * np.sin(.7)])
    assert (y[4:] == [5, 6]).all()
    y = oracle.rotate(x, [7], rope, interleaved=True)[0, 0]
    assert np.allclose(y[:2], [np.cos(7) - 2 * np.sin(7), 2 * np.cos(7) + np.sin(7)])
    assert np.allclose(y[2:4], [3 * np.cos(.7) - 4 * np.sin(.7), 4 * np.cos(.7) + 3 * np.sin(.7)])
    # a product depends on the positions' difference only
    rng = np.random.default_rng(3)
    a, b = rng.normal(size=(1, 1, 8)), rng.normal(size=(1, 1, 8))
    rope = oracle.rope_table(40, 8)
    dots = [np.sum(oracle.rotate(a, [i + 5], rope) * oracle.rotate(b, [i], rope)) for i in (0, 3, 30)]
    assert np.allclose(dots, dots[0])


def test_oracle_block_scale():
    assert oracle.block_scale(0.0) == 0.0
    assert oracle.block_scale(448.0) == 1.0
    assert oracle.block_scale(np.nextafter(448.0, 500)) == 2.0
    assert oracle.block_scale(1.75 * 2.0 ** -9) == 2.0 ** -17
    assert oracle.block_scale(1e-44) == 2.0 ** -126


def test_oracle_paged_equals_dense():
    """The paged append and decode against a dense cache decoded by the ring
    oracle (a ring that never wraps holds positions in order)."""
    rng = np.random.default_rng(5)
    lens = np.array([0, 1, 16, 50])
    n, page, mp = len(lens), 16, 4
    table = rng.permutation(n * mp + 2)[: n * mp].reshape(n, mp)
    k, v = rng.normal(size=(2, lens.sum(), Hkv, 8))
    cu = np.concatenate([[0], np.cumsum(lens)])
    kp = np.full((n * mp + 2, Hkv, page, 8), 9.0)
    kp, vp = oracle.paged_append(k, v, table, lens, kp, kp, cu)
    q, sink = rng.normal(size=(n, Hq, 8)), rng.normal(size=Hq)
    kd, vd = np.zeros((2, n, 64, Hkv, 8))
    for b in range(n):
        kd[b, : lens[b]], vd[b, : lens[b]] = k[cu[b]:cu[b + 1]], v[cu[b]:cu[b + 1]]
    want = oracle.decode(q, kd, vd, lens.astype(np.int32), 0, 64, sink, 0.3)
    got = oracle.paged_decode(q, kp, vp, table, lens, 0, 0, sink, 0.3)
    for a, b in zip(got, want):
        assert np.allclose(a, b, atol=1e-12)
    # a window with sink tokens against the band's rows of the dense forward
    L = 50
    rows = np.array([[L - 1, h] for h in range(Hq)], dtype=np.int32)
    qq = np.zeros((L, Hq, 8)); qq[L - 1] = q[3]
    ro, rl, rs = oracle.fwd_rows(qq, k[cu[3]:], v[cu[3]:], sink, 0.3, rows, causal=True, n_sink=3,
                                 window=20, cu_seqlens=torch.tensor([0, L], dtype=i32))
    go, gl, gs = oracle.paged_decode(q, kp, vp, table, lens, 3, 20, sink, 0.3)
    assert np.allclose(go[3], ro) and np.allclose(gl[3], rl) and np.allclose(gs[3], rs)


def test_oracle_fp8_append_growth():
    """A block's scale grows with a larger new row, its earlier codes keep their
    values where the format holds them, and a smaller row leaves it alone."""
    table, lens = np.array([[1]]), np.array([2])
    codes, scale = np.full((2, 1, 16, 8), 0x7F, np.uint8), np.full((2, 1), 5.0)
    x = np.zeros((2, 1, 8))
    x[0, 0, :3] = [448, 1.0, 2.0 ** -9]
    x[1, 0, :2] = [-3, np.inf]
    codes, scale = oracle.paged_append_fp8(x, table, lens, codes, scale, np.array([0, 2]))
    assert scale[1, 0] == 1.0 and scale[0, 0] == 5.0
    assert (oracle.fp8_e4m3_value(codes[1, 0, 0, :3]) == [448, 1, 2.0 ** -9]).all()
    assert (oracle.fp8_e4m3_value(codes[1, 0, 1, :2]) == [-3, 448]).all()
    y = np.full((1, 1, 8), 1000.0)
    codes, scale = oracle.paged_append_fp8(y, table, np.array([3]), codes, scale)
    assert scale[1, 0] == 4.0
    assert (4 * oracle.fp8_e4m3_value(codes[1, 0, 0, :3]) == [448, 1, 0]).all()
    assert (4 * oracle.fp8_e4m3_value(codes[1, 0, 2]) == 1024).all()  # 250 -> 256
    codes, scale = oracle.paged_append_fp8(y * 0 + 1, table, np.array([4]), codes, scale)
    assert scale[1, 0] == 4.0 and (4 * oracle.fp8_e4m3_value(codes[1, 0, 3]) == 1).all()
