"""Host-side refusals of the rotation and of the paged cache's calls (none
reaches the GPU), and the plain forms that their GPU tests rest on."""
import ctypes

import numpy as np
import pytest
import torch

import hierarchical_routed_sparse_b200 as hga
from hierarchical_routed_sparse_b200 import binding as B
from hierarchical_routed_sparse_b200 import build as hbuild

import paged_ref as R

P16 = ctypes.c_void_p(16)
BAD, UNSUP = hga.HGA_ERR_INVALID_ARG, hga.HGA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    hbuild.build()
    return hga.load()


def _paged(**kw):
    base = dict(B=2, Hq=8, Hkv=2, d=128, n_pages=16, max_chunks=8, k_c=4, k_g=16)
    base.update(kw)
    return hga.PagedParams(**base)


@pytest.mark.parametrize("kw,code", [
    (dict(d=96), UNSUP), (dict(B=0), BAD), (dict(Hq=7), BAD), (dict(n_pages=0), BAD), (dict(n_pages=1 << 31), BAD),
    (dict(max_chunks=0), BAD), (dict(max_chunks=1 << 30), UNSUP), (dict(k_c=0), BAD), (dict(k_g=-7), BAD),
    (dict(dtype=2), BAD), (dict(cache_dtype=0), BAD), (dict(scale=float("inf")), BAD), (dict(scale=-1.0), BAD),
    (dict(k_c=1 << 30), UNSUP), (dict(B=1 << 24, Hkv=8), UNSUP),
])
def test_paged_params_are_refused(lib, kw, code):
    p = _paged(**kw).c()
    wc, wg = ctypes.c_int(), ctypes.c_int()
    assert lib.hga_paged_widths(ctypes.byref(p), ctypes.byref(wc), ctypes.byref(wg)) == code
    assert lib.hga_last_error().decode()
    c = B._PagedCache(*[16] * 9)
    assert lib.hga_paged_decode(ctypes.byref(p), ctypes.byref(c), P16, P16, P16, P16, P16, P16, P16, 1 << 40, None) == code
    assert _append(lib, p, c) == code


def _append(lib, p, c, pos=P16, cu=P16, N=5, q=P16, qs=(1024, 128), k=P16, ks=(256, 128), v=P16, vs=(256, 128),
            out=P16, rope=P16, rows=100, rot=128, inter=0):
    return lib.hga_paged_append(ctypes.byref(p), None if c is None else ctypes.byref(c), pos, cu, N, q, *qs, k, *ks, v, *vs, out,
                                rope, rows, rot, inter, None)


def test_paged_widths(lib):
    assert hga.paged_widths(_paged()) == (4, 16)
    assert hga.paged_widths(_paged(k_c=hga.HGA_ALL, k_g=hga.HGA_ALL)) == (8, 64)
    assert hga.paged_widths(_paged(k_g=hga.HGA_ALL)) == (4, 32)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), BAD), (dict(cu=None, N=5), BAD), (dict(rot=24), BAD), (dict(rot=144), BAD), (dict(rot=-16), BAD),
    (dict(rope=None), BAD), (dict(rope=ctypes.c_void_p(24)), BAD), (dict(rows=0), BAD), (dict(ks=(4, 128)), BAD),
    (dict(vs=(256, -128)), BAD), (dict(qs=(1024, 3)), BAD), (dict(q=None), BAD), (dict(out=None), BAD),
    (dict(k=None), BAD), (dict(v=ctypes.c_void_p(8)), BAD), (dict(pos=None), BAD), (dict(q=ctypes.c_void_p(2)), BAD),
    (dict(out=ctypes.c_void_p(2)), BAD), (dict(c=None), BAD),
])
def test_append_refusals(lib, kw, code):
    kw = dict(kw)
    c = kw.pop("c", B._PagedCache(*[16] * 9))
    assert _append(lib, _paged().c(), c, **kw) == code
    assert lib.hga_last_error().decode()


@pytest.mark.parametrize("i", range(9))
def test_cache_pointers_are_checked(lib, i):
    for bad in (0, 24):
        ptr = [16] * 9
        ptr[i] = bad
        c, p = B._PagedCache(*ptr), _paged().c()
        assert _append(lib, p, c) == BAD
        assert lib.hga_paged_decode(ctypes.byref(p), ctypes.byref(c), P16, P16, P16, P16, P16, P16, P16, 1 << 40, None) == BAD


def test_append_of_nothing_is_a_no_op(lib):
    assert _append(lib, _paged().c(), B._PagedCache(*[16] * 9), N=0) == hga.HGA_OK


def test_decode_refusals(lib):
    c = B._PagedCache(*[16] * 9)

    def call(p, pos=P16, q=P16, O=P16, lse=P16, cidx=P16, gidx=P16, ws=P16, n=1 << 40):
        return lib.hga_paged_decode(ctypes.byref(p.c()), ctypes.byref(c), pos, q, O, lse, cidx, gidx, ws, n, None)

    for name in ("pos", "q", "O", "lse", "cidx", "gidx"):
        assert call(_paged(), **{name: None}) == BAD, name
    assert call(_paged(k_c=hga.HGA_ALL, k_g=hga.HGA_ALL), cidx=None) == BAD       # one without the other
    assert call(_paged(k_c=hga.HGA_ALL), cidx=None, gidx=None) == BAD
    dense = _paged(k_c=hga.HGA_ALL, k_g=hga.HGA_ALL)
    need = hga.paged_workspace_size(dense)
    assert need > 0 and hga.paged_workspace_size(_paged()) == 0
    assert call(dense, cidx=None, gidx=None, n=need - 1) == BAD
    assert call(dense, cidx=None, gidx=None, ws=None) == BAD
    assert call(_paged(k_c=hga.HGA_ALL, k_g=hga.HGA_ALL, B=1 << 12, max_chunks=1 << 18), cidx=None, gidx=None) == UNSUP
    assert call(dense, cidx=None, gidx=None, ws=ctypes.c_void_p(4)) == BAD
    assert call(_paged(Hq=18, Hkv=2)) == UNSUP                                    # 9 q-heads per kv-head
    assert call(_paged(k_c=1 << 14, max_chunks=1 << 14)) == UNSUP                 # routing state past shared memory


def _rope(**kw):
    base = dict(B=2, H=4, d=128, rot_dim=128, interleaved=0, x_dtype=1, y_dtype=0, T=10, pos0=5, table_rows=15,
                x_batch=10 * 512, x_token=512, x_head=128)
    base.update(kw)
    return B._RopeParams(*[base[n] for n, _ in B._RopeParams._fields_])


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), BAD), (dict(H=0), BAD), (dict(d=32), UNSUP), (dict(x_dtype=2), BAD), (dict(y_dtype=-1), BAD),
    (dict(T=-1), BAD), (dict(pos0=-1), BAD), (dict(T=11), BAD), (dict(rot_dim=8), BAD), (dict(rot_dim=256), BAD),
    (dict(x_head=2), BAD), (dict(x_token=-512), BAD), (dict(T=1 << 31), BAD), (dict(H=1 << 20, B=1), UNSUP),
])
def test_rope_refusals(lib, kw, code):
    p = _rope(**kw)
    for f in (lib.hga_rope_fwd, lib.hga_rope_bwd):
        assert f(ctypes.byref(p), P16, P16, P16, None) == code
        assert lib.hga_last_error().decode()


def test_gradient_rows_must_not_share_elements(lib):
    for kw in (dict(x_head=0), dict(x_token=64), dict(x_batch=0)):
        p = _rope(**kw)
        assert lib.hga_rope_bwd(ctypes.byref(p), P16, P16, P16, None) == BAD
        assert lib.hga_rope_fwd(ctypes.byref(p), None, P16, P16, None) == BAD     # (refused for the pointer: fwd may repeat rows)
        assert "overlap" not in lib.hga_last_error().decode()


def test_rope_pointer_refusals(lib):
    p = _rope()
    for a in ((None, P16, P16), (P16, None, P16), (P16, P16, None), (ctypes.c_void_p(4), P16, P16),
              (P16, ctypes.c_void_p(4), P16), (P16, P16, ctypes.c_void_p(4))):
        assert lib.hga_rope_fwd(ctypes.byref(p), *a, None) == BAD
    empty = _rope(T=0)
    assert lib.hga_rope_fwd(ctypes.byref(empty), None, P16, None, None) == hga.HGA_OK


def test_python_refusals_and_no_cpu_fallback(lib):
    x, y, t = torch.zeros(1, 4, 2, 64), torch.zeros(1, 2, 4, 64), torch.zeros(4, 64)
    with pytest.raises(ValueError):
        hga.rope_fwd(x, y, t)                                  # host tensors
    with pytest.raises(ValueError):
        hga.rope_fwd(x, y[:, :, :3], t)
    with pytest.raises(ValueError):
        hga.rope_fwd(x.half(), y, t)
    with pytest.raises(ValueError):
        hga.rope_fwd(x, y, t.double())
    with pytest.raises(ValueError):
        hga.rope_table(4, 24)
    with pytest.raises(ValueError):
        hga.PagedCache(_paged(), device="cpu")                 # host tensors
    with pytest.raises(ValueError):
        hga.PagedCache(_paged(), k_rows=torch.zeros(1))


def test_structs_match_the_header(lib, tmp_path):
    import os
    import subprocess
    src = tmp_path / "s.c"
    src.write_text('#include "hga.h"\n#include <stdio.h>\nint main(void){printf("%zu %zu %zu\\n", sizeof(hga_rope_params),'
                   ' sizeof(hga_paged_params), sizeof(hga_paged_cache)); return 0;}\n')
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run(["gcc", "-I", inc, str(src), "-o", str(tmp_path / "s")], check=True)
    got = subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in got] == [ctypes.sizeof(t) for t in (B._RopeParams, B._PagedParams, B._PagedCache)]


def test_plain_e4m3_agrees_with_torch():
    x = torch.linspace(-448, 448, 4001).float()
    x = torch.cat([x, x / 448, x / 448 * 2.0 ** -7, torch.tensor([0.0, 2.0 ** -10, 2.0 ** -9, 3 * 2.0 ** -10])])
    np.testing.assert_array_equal(R.e4m3_code(x.numpy()), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    codes = torch.arange(256, dtype=torch.uint8)
    np.testing.assert_array_equal(R.E4M3, codes.view(torch.float8_e4m3fn).double().numpy())


@pytest.mark.parametrize("cache", ["int8", "e4m3"])
def test_plain_quantisation_is_within_half_a_step(cache):
    x = np.random.default_rng(1).standard_normal((50, 8, 64)).astype(np.float32)
    x[0] *= 1e-42                                              # below the smallest scale
    x[1] = 0
    x[2] *= 1e30
    code, scale = R.quantise(x, cache)
    err = np.abs(R.held(code, scale, cache) - x)
    step = 0.5 * (1 + 2e-4) if cache == "int8" else 2.0 ** -10
    tol = step * scale[:, None, None].astype(np.float64) + (0 if cache == "int8" else 2.0 ** -4 * (1 + 2e-6) * np.abs(x))
    assert (err <= tol).all()


def test_advance_refusals(lib):
    def call(p=None, pos=P16, cu=P16, N=5, rows=100, rot=128, last=ctypes.c_void_p(32)):
        return lib.hga_paged_advance(ctypes.byref((p or _paged()).c()), pos, cu, N, rows, rot, last, None)

    for kw, code in ((dict(pos=None), BAD), (dict(N=-1), BAD), (dict(N=1 << 31), BAD), (dict(cu=None), BAD), (dict(rot=24), BAD),
                     (dict(rot=144), BAD), (dict(rows=0), BAD), (dict(last=P16), BAD), (dict(p=_paged(d=96)), UNSUP),
                     (dict(p=_paged(B=0)), BAD)):
        assert call(**kw) == code, kw
        assert lib.hga_last_error().decode()
    assert lib.hga_paged_advance(None, P16, None, 2, 1, 0, None, None) == BAD


def test_a_generation_state_needs_a_long_enough_table(lib):
    for tokens, rope in ((129, torch.zeros(128, 64)), (0, None), (64, torch.zeros(64, 64).double())):
        with pytest.raises(ValueError, match="rope|rotation|max_tokens"):       # before any device tensor is made
            hga.PagedDecodeState(1, 4, 2, 64, tokens, 2, 9, rope=rope)
