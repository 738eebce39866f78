"""Decode from the paged cache, and its summaries, over the range of finite
floats: values, scores, queries and keys near its ends.

Where scores are moderate the bound is that of test_gpu_paged.  Where they are
so far apart that the highest key takes all the weight (its lead, in float64,
is asserted to exceed both keys' errors by far more than a weight's last bit),
O is that key's value and lse its score, each to 2^-20 (a weight's two parts,
its exponential, the sums).
"""
import math

import numpy as np
import pytest
import torch

import hierarchical_routed_sparse_b200 as hga

import paged_ref as R
from test_gpu_paged import TENSORS, Plain, _cache, _check_decode, _decode, _filled, _int32, _params, _snapshot

pytestmark = pytest.mark.gpu
KINDS = [("bf16", "int8", 128), ("fp32", "e4m3", 64), ("fp32", "int8", 64), ("bf16", "e4m3", 128)]


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from hierarchical_routed_sparse_b200 import build
    build.build()
    hga.load()
    hga.device_check(clear=True)


def _both(p, kind, c, pos, q):
    """The decode call in its routed form and over the whole cache."""
    _check_decode(c, kind, pos, q, _decode(c, pos, q))
    whole = hga.PagedParams(p.B, p.Hq, p.Hkv, p.d, p.n_pages, p.max_chunks, -1, -1, p.dtype, p.cache_dtype)
    w = hga.PagedCache(whole, **{n: getattr(c, n) for n in TENSORS + ("table",)})
    _check_decode(w, kind, pos, q, _decode(w, pos, q, rows=False), rows=False)


@pytest.mark.parametrize("dtype,kind,d", KINDS)
@pytest.mark.parametrize("power", [-85, 60, 101, 104, 112, 124])
def test_values_of_every_size(power, dtype, kind, d):
    # Value scales up to 2^119, values up to 2^126: finite, as append holds them.
    p = _params(2, 8, 2, d, 24, 11, dtype, kind, 3, 13)
    c, q = _filled(p, kind, [640, 300])
    c.v_scale *= 2.0 ** power
    c.v_tail.copy_(c.v_tail.float() * 2.0 ** power)
    assert float(c.v_tail[0, :, :64].float().abs().max()) < 3e38
    _both(p, kind, c, [639, 299], q)


@pytest.mark.parametrize("dtype,kind,d", KINDS)
@pytest.mark.parametrize("power", [10, 30, 45, 100, 120])
@pytest.mark.parametrize("zero", [0, 1])
def test_groups_of_zeros_beside_large_values(zero, power, dtype, kind, d):
    # Every other chunk holds zeros (with the smallest scale, as append writes it):
    # its keys count in the normaliser as much as those of large values.
    p = _params(2, 4, 1, d, 45, 22, dtype, kind, 8, 60)
    c, q = _filled(p, kind, [1300, 333])
    c.v_scale *= 2.0 ** power
    c.v_tail.copy_(c.v_tail.float() * 2.0 ** power)
    for b, n in ((0, 20), (1, 5)):
        pages = c.table[b, zero:n:2].long()
        c.v_pages.view(torch.uint8)[pages] = 0
        c.v_scale[pages] = 2.0 ** -126
    _both(p, kind, c, [1299, 332], q)


def _one_takes_all(c, kind, b, q, got_O, got_lse, pos):
    """Heads of sequence b (one kv-head, whole cache) against the highest key."""
    p = c.p
    c0 = pos // 64
    pages = c.table[b, :c0].long()
    u8 = lambda t: t[pages].view(torch.uint8).cpu().numpy().reshape(c0, 8, 8, p.d)  # noqa: E731
    k, v = (np.concatenate([R.held(u8(codes), scale[pages, 0].cpu().numpy(), kind).reshape(-1, p.d),
                            tail[b, 0, :pos % 64 + 1].double().cpu().numpy()])
            for codes, scale, tail in ((c.k_pages, c.k_scale, c.k_tail), (c.v_pages, c.v_scale, c.v_tail)))
    qd = q[b].double().cpu().numpy()
    s = qd @ k.T / math.sqrt(p.d)
    err = (p.d + 8) * 2.0 ** -24 / math.sqrt(p.d) * (np.abs(qd) @ np.abs(k).T).max(1)
    order = np.argsort(-s, 1)
    heads = np.arange(len(s))
    if s.shape[1] > 1:
        assert (s[heads, order[:, 0]] - s[heads, order[:, 1]] > 4 * err + 100).all()
    assert np.abs(got_O - v[order[:, 0]]).max() <= 2.0 ** -20 * np.abs(v).max()
    assert (np.abs(got_lse - s[heads, order[:, 0]]) <= err + 2.0 ** -20 * (1 + np.abs(s).max())).all()


@pytest.mark.parametrize("dtype,kind,d", KINDS)
@pytest.mark.parametrize("power", range(22, 32))
@pytest.mark.parametrize("values", [0, 10])
def test_scores_past_the_integers_of_float32(values, power, dtype, kind, d):
    # Scores at which float32 steps by 1 to 512: a reference that is not itself a
    # score is off by whole powers of two.
    p = _params(1, 4, 1, d, 12, 10, dtype, kind)
    c, q = _filled(p, kind, [600], seed=1)
    q = (q.float() * 2.0 ** power).to(q.dtype)
    c.v_scale *= 2.0 ** values
    c.v_tail.copy_(c.v_tail.float() * 2.0 ** values)
    for rows in (False, True):
        O, lse, _, _ = _decode(c, [599], q, rows=rows)
        _one_takes_all(c, kind, 0, q, O[0], lse[0], 599)


@pytest.mark.parametrize("dtype,kind,d", KINDS)
@pytest.mark.parametrize("power", [95, 104, 114])
@pytest.mark.parametrize("n", [1, 40, 300])
def test_every_score_far_below_zero(n, power, dtype, kind, d):
    # All keys against the query: the highest score is still below -2^95.
    p = _params(1, 4, 1, d, 8, 5, dtype, kind)
    c, q = _filled(p, kind, [n], seed=3)
    q = (q.float().abs() * 2.0 ** power).to(q.dtype)
    codes = c.k_pages.view(torch.uint8)
    codes.copy_(torch.where(codes < 128, 256 - codes.int(), codes.int()).byte() if kind == "int8" else codes | 128)
    c.k_tail.copy_(-c.k_tail.abs())
    for rows in (False, True):
        O, lse, _, _ = _decode(c, [n - 1], q, rows=rows)
        assert (lse < -2.0 ** power).all()
        _one_takes_all(c, kind, 0, q, O[0], lse[0], n - 1)


@pytest.mark.parametrize("dtype,kind,d", KINDS)
@pytest.mark.parametrize("power", [60, 100, 112, 118])
def test_small_queries_of_large_keys(power, dtype, kind, d):
    # Scores of ordinary size from queries of 2^-118 and keys of 2^118.
    p = _params(2, 8, 2, d, 24, 11, dtype, kind, 3, 13)
    c, q = _filled(p, kind, [640, 300], seed=5)
    q = (q.float() * 2.0 ** -power).to(q.dtype)
    for t in (c.k_scale, c.k_tail, c.csum, c.gsum):
        t *= 2.0 ** power
    _both(p, kind, c, [639, 299], q)


@pytest.mark.parametrize("dtype,kind,d", KINDS)
@pytest.mark.parametrize("power", [0, 121, 124, 126])
def test_summaries_of_the_largest_keys(power, dtype, kind, d):
    # Keys of one sign whose sums over a group (from 2^125 on) or a chunk (from
    # 2^122) are past float32, while their means are not; codes, scales and open
    # rows as everywhere.
    p = _params(1, 4, 2, d, 4, 3, dtype, kind, 1, 5)
    c = _cache(p)
    plain, before = Plain(p, kind, c.table), _snapshot(c)
    g = torch.Generator().manual_seed(power)
    k = ((1 + torch.rand(130, 2, d, generator=g)) * 2.0 ** power).to(p.torch_dtype).cuda()
    v = torch.randn(130, 2, d, generator=g).to(p.torch_dtype).cuda()
    at = 0
    for n in (60, 66, 4):
        c.append(_int32([at]), k[at:at + n], v[at:at + n], cu=_int32([0, n]))
        at += n
    torch.cuda.synchronize()
    plain.append(0, k, v, None, False)
    plain.check(c, before)
    q = (torch.randn(1, 4, d, generator=g) * 2.0 ** -min(power, 118)).to(p.torch_dtype).cuda()
    _both(p, kind, c, [129], q)
    assert hga.device_check() == 0


def test_a_workspace_that_is_not_contiguous_is_refused():
    # As many bytes by its shape as are needed, and far fewer behind its pointer.
    p = _params(1, 4, 2, 64, 4, 3, "bf16", "int8")
    c, q = _filled(p, "int8", [100])
    n = hga.paged_workspace_size(p)
    O, lse = torch.full((1, 4, 64), 9.0, device="cuda"), torch.full((1, 4), 9.0, device="cuda")
    for ws in (torch.empty(16, dtype=torch.uint8, device="cuda")[:1].expand(n),
               torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError, match="contiguous"):
            c.decode(_int32([99]), q, O, lse, workspace=ws)
    torch.cuda.synchronize()
    assert (O == 9.0).all()
    c.decode(_int32([99]), q, O, lse, workspace=torch.empty(n // 4, dtype=torch.float32, device="cuda"))
    _check_decode(c, "int8", [99], q, (O.cpu().numpy(), lse.cpu().numpy(), None, None), rows=False)
