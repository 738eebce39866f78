"""The rotation inside the segment layer (segment.RotaryHeads): two segments
with all-routing against a dense masked softmax in float32 with the same
rotation, and the rotation's gradient against difference quotients.

Both sides round q, k (after the rotation), v and the attention's upstream
gradient to the activations' type, so they differ by float32 sums and by
values that a rounding puts on the other side of a bf16 step; those are rare
and their parts of a weight gradient average out: the bound is the one that
the layer without rotation is held to.
"""
import math

import pytest
import torch

import hierarchical_routed_sparse_b200 as hga
from hierarchical_routed_sparse_b200.segment import HGASegmentLayer, RotaryHeads, run_tbptt

from test_gpu_segment import _GradCast, _round

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from hierarchical_routed_sparse_b200 import build
    build.build()
    hga.load()


def _turn(x, rows, interleaved):
    """x [B][T][H][d] by table rows [T][rot], in elementary torch operations."""
    rot = rows.shape[-1]
    h = rot // 2
    c, s = rows[:, None, :h], rows[:, None, h:]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :h], x[..., h:rot])
    ya, yb = a * c - b * s, b * c + a * s
    y = torch.stack([ya, yb], -1).flatten(-2) if interleaved else torch.cat([ya, yb], -1)
    return torch.cat([y, x[..., rot:]], -1)


@pytest.mark.parametrize("dtype,d,rot,inter", [(torch.bfloat16, 128, 128, False), (torch.float32, 64, 32, True)],
                         ids=["bf16_half_split", "fp32_interleaved_partial"])
def test_layer_with_rotation(dtype, d, rot, inter):
    torch.manual_seed(3)
    d_model, Hq, Hkv, seg, T, Bn = 96, 4, 2, 128, 256, 2
    rope = hga.rope_table(T, rot)
    layer = HGASegmentLayer(d_model, Hq, Hkv, d, k_c=hga.HGA_ALL, k_g=hga.HGA_ALL, dtype=dtype, rope=rope, interleaved=inter)
    x, target = torch.randn(Bn, T, d_model, device="cuda"), torch.randn(Bn, T, d_model, device="cuda")
    run_tbptt(layer, x, target, seg)
    got = {n: p.grad.clone() for n, p in layer.named_parameters()}
    for p in layer.parameters():
        p.grad = None
    Kh = Vh = None
    for s in range(0, T, seg):
        xs = x[:, s:s + seg]
        rows = rope[s:s + seg]
        q = _round(_turn(layer.wq(xs).view(Bn, seg, Hq, d), rows, inter).transpose(1, 2), dtype)
        k = _round(_turn(layer.wk(xs).view(Bn, seg, Hkv, d), rows, inter).transpose(1, 2), dtype)
        v = _round(layer.wv(xs).view(Bn, seg, Hkv, d).transpose(1, 2), dtype)
        K, V = (k, v) if Kh is None else (torch.cat([Kh, k], 2), torch.cat([Vh, v], 2))
        S = torch.einsum("bhid,bhtd->bhit", q, K.repeat_interleave(Hq // Hkv, 1)) / math.sqrt(d)
        seen = torch.arange(s + seg, device="cuda")[None] <= s + torch.arange(seg, device="cuda")[:, None]
        P = torch.softmax(S.masked_fill(~seen, float("-inf")), -1)
        O = _GradCast.apply(torch.einsum("bhit,bhtd->bhid", P, V.repeat_interleave(Hq // Hkv, 1)), dtype)
        out = layer.wo(O.transpose(1, 2).reshape(Bn, seg, Hq * d))
        (0.5 * (out - target[:, s:s + seg]).pow(2).mean()).backward()
        Kh, Vh = K.detach(), V.detach()
    for n, p in layer.named_parameters():
        rel = float((got[n] - p.grad).norm() / p.grad.norm())
        assert rel < 2e-3, f"{n}: relative gradient error {rel:.3g}"


def test_gradient_against_differences():
    # y is linear in x, so the quotient over a step of 1 is exact up to the
    # outputs' roundings (2^-23 of sums of some 2000 terms around 1).
    torch.manual_seed(4)
    table = hga.rope_table(40, 64)
    x = torch.randn(1, 30, 2, 64, device="cuda", requires_grad=True)
    w = torch.randn(1, 2, 30, 64, device="cuda")
    RotaryHeads.apply(x, table, 7, False, torch.float32).backward(w)
    with torch.no_grad():
        base = RotaryHeads.apply(x, table, 7, False, torch.float32).double()
        for t, h, e in ((0, 0, 0), (29, 1, 63), (13, 0, 32), (5, 1, 31)):
            step = x.clone()
            step[0, t, h, e] += 1
            diff = ((RotaryHeads.apply(step, table, 7, False, torch.float32).double() - base) * w.double()).sum()
            assert abs(float(diff) - float(x.grad[0, t, h, e])) <= 16 * 2.0 ** -23 * float(w.abs().max()) * 4


def test_positions_past_the_table_are_refused():
    layer = HGASegmentLayer(64, 2, 1, 64, rope=hga.rope_table(100, 64))
    with pytest.raises(hga.HGAError):
        layer.segment(torch.randn(1, 128, 64, device="cuda"))


def test_a_second_derivative_is_refused():
    x = torch.randn(1, 8, 1, 64, device="cuda", requires_grad=True)
    y = RotaryHeads.apply(x, hga.rope_table(8, 64), 0, False, torch.float32)
    dx, = torch.autograd.grad((y ** 3).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dx.sum().backward()


def test_gradient_captured_and_replayed():
    # Forward and gradient in one graph, replayed on other values.  (With an
    # eager graph of the same leaf alive PyTorch's own stream bookkeeping
    # invalidates any capture of a gradient, whatever the function.)
    table = hga.rope_table(200, 64)
    x = torch.randn(2, 150, 3, 64, device="cuda", requires_grad=True)
    w = torch.randn(2, 3, 150, 64, device="cuda")
    run = lambda: torch.autograd.grad(RotaryHeads.apply(x, table, 50, True, torch.bfloat16), x, w.bfloat16())[0]  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dx = run()
    with torch.no_grad():
        w.normal_()
    dx.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(dx, run())
