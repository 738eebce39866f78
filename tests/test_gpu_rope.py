"""The position rotation (hga_rope_fwd / hga_rope_bwd) against plain numpy.

float32 outputs equal the definition's own operations (each product and sum
rounded to float32) bit for bit; against float64 an element of a pair is off
by at most three roundings of the pair's products, 3 * 2^-24 (|x1| + |x2|);
a bf16 output adds half a bf16 step, 2^-8 relative to the value."""
import numpy as np
import pytest
import torch

import hierarchical_routed_sparse_b200 as hga

from paged_ref import rotate

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from hierarchical_routed_sparse_b200 import build
    build.build()
    hga.load()


def _check(got, x, rows, inter, back, out):
    """got, x as [..., d] with matching table rows."""
    exact = rotate(x.astype(np.float64), rows.astype(np.float64), inter, back)
    f32 = rotate(x.astype(np.float32), rows, inter, back)
    if out == "fp32":
        np.testing.assert_array_equal(got, f32)
    rot = rows.shape[-1]
    pair = np.abs(x).astype(np.float64)
    if rot:
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
        both = pair[..., a] + pair[..., b]
        pair[..., a] = pair[..., b] = both
    tol = 3 * 2.0 ** -24 * pair
    if out == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(exact) + tol)
    assert (np.abs(got - exact) <= tol).all(), float((np.abs(got - exact) - tol).max())


CASES = [  # B, T, H, d, rot, interleaved, pos0, x, y
    (1, 1, 1, 64, 64, False, 0, "fp32", "fp32"),
    (2, 33, 5, 128, 128, False, 7, "fp32", "bf16"),
    (1, 64, 4, 128, 128, True, 100000, "bf16", "fp32"),
    (3, 65, 7, 64, 32, True, 3, "bf16", "bf16"),
    (2, 31, 9, 128, 16, False, 50, "fp32", "fp32"),
    (1, 130, 3, 64, 48, False, 1, "fp32", "bf16"),
    (2, 20, 2, 128, 0, False, 0, "fp32", "bf16"),
]


@pytest.mark.parametrize("back", [False, True], ids=["fwd", "bwd"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_rotation(case, back):
    B, T, H, d, rot, inter, pos0, xt, yt = case
    g = torch.Generator().manual_seed(B * 100 + T)
    table = hga.rope_table(pos0 + T, rot) if rot else None
    rows = (table.cpu().numpy()[pos0:pos0 + T] if rot else np.zeros((T, 0), np.float32))
    wide = torch.randn(B, T, H + 2, d, generator=g).to(DT[xt]).cuda()   # projections next to each other
    x = wide[:, :, 1:H + 1]
    y = torch.full((B, H, T, d), 7.0, dtype=DT[yt], device="cuda")
    if not back:
        hga.rope_fwd(x, y, table, pos0=pos0, interleaved=inter)
        got = y.float().cpu().numpy()
        _check(got, x.float().cpu().numpy().transpose(0, 2, 1, 3), rows, inter, False, yt)
        return
    dy = torch.randn(B, H, T, d, generator=g).to(DT[yt]).cuda()
    before = wide.clone()
    hga.rope_bwd(dy, x, table, pos0=pos0, interleaved=inter)
    _check(x.float().cpu().numpy(), dy.float().cpu().numpy().transpose(0, 2, 1, 3), rows[:, None], inter, True, xt)
    assert torch.equal(wide[:, :, 0], before[:, :, 0]) and torch.equal(wide[:, :, H + 1], before[:, :, H + 1])


def test_gradient_is_the_transpose():
    # <R x, z> = <x, R^T z> and, R being linear, the difference quotient
    # (R(x + e) - R(x)) = R e: both in float64 sums of float32 outputs.
    B, T, H, d = 2, 40, 3, 128
    table = hga.rope_table(T + 5, 64)
    x, z = torch.randn(B, T, H, d, device="cuda"), torch.randn(B, H, T, d, device="cuda")
    y, dx = torch.empty(B, H, T, d, device="cuda"), torch.empty(B, T, H, d, device="cuda")
    hga.rope_fwd(x, y, table, pos0=5)
    hga.rope_bwd(z, dx, table, pos0=5)
    left = float((y.double() * z.double()).sum())
    right = float((x.double() * dx.double()).sum())
    size = float((y.abs().double() * z.abs().double()).sum())
    assert abs(left - right) <= 2 * 3 * 2.0 ** -24 * 2 * size
    back = torch.empty_like(x)
    hga.rope_bwd(y, back, table, pos0=5)           # a rotation: R^T R x = x
    assert float((back - x).abs().max()) <= 12 * 2.0 ** -24 * 2 * float(x.abs().max())


def test_transposed_input_and_another_stream():
    x = torch.randn(2, 6, 50, 64, device="cuda")    # [B][H][T][d] memory seen as [B][T][H][d]
    table = hga.rope_table(50, 64)
    y = torch.empty(2, 6, 50, 64, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        hga.rope_fwd(x.transpose(1, 2), y, table)
    s.synchronize()
    _check(y.cpu().numpy(), x.cpu().numpy(), table.cpu().numpy(), False, False, "fp32")


def test_captured_and_replayed():
    x, table = torch.randn(1, 70, 4, 128, device="cuda"), hga.rope_table(70, 128)
    y = torch.empty(1, 4, 70, 128, device="cuda", dtype=torch.bfloat16)
    hga.rope_fwd(x, y, table)
    want = y.clone()
    y.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hga.rope_fwd(x, y, table)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_strides_of_dimensions_of_one_do_not_matter():
    # What such a stride says is nobody's offset (a view made by permute may have
    # any): contiguous rows are taken, by the rotation and by the append.
    g = torch.Generator().manual_seed(11)
    x = torch.randn(5, 3, 64, 1, generator=g).cuda().permute(3, 0, 1, 2)        # [1][5][3][64], batch stride 1
    assert x.is_contiguous() and x.stride(0) == 1
    rope = hga.rope_table(16, 64)
    want, got = torch.empty(1, 3, 5, 64, device="cuda"), torch.empty(1, 3, 5, 64, device="cuda")
    hga.rope_fwd(x.clone(memory_format=torch.contiguous_format).view(1, 5, 3, 64).as_strided((1, 5, 3, 64), (960, 192, 64, 1)), want, rope)
    hga.rope_fwd(x, got, rope)
    assert torch.equal(got, want)
    back = torch.empty(960, device="cuda").as_strided((1, 5, 3, 64), (1, 192, 64, 1))
    hga.rope_bwd(want, back, rope)
    assert float((back - x).abs().max()) < 1e-5
    one = torch.randn(64, generator=g).bfloat16().cuda().as_strided((1, 1, 64), (3, 1, 1))
    p = hga.PagedParams(1, 1, 1, 64, 1, 1)
    caches = [hga.PagedCache(p) for _ in range(2)]
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    for c, k in zip(caches, (one, one.clone().view(64).view(1, 1, 64))):
        out = torch.empty(1, 1, 64, dtype=torch.bfloat16, device="cuda")
        c.append(zero, k, k, q=k, q_out=out, rope=rope)
        assert torch.equal(c.v_tail[0, 0, 0], one.view(64))
    assert torch.equal(caches[0].k_tail, caches[1].k_tail)
