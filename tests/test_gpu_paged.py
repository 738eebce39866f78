"""The paged 8-bit cache (hga_paged_append, hga_paged_decode) against plain
numpy (paged_ref.py).

append: rotated keys, codes and scales equal the definition's float32
operations bit for bit; summaries are float32 means of at most 64 values, off
by at most 64 * 2^-24 times the mean of the magnitudes.

decode: routing rows equal those of float64 scores exactly.  A float32 score
over d products is off by at most e = (d + 8) 2^-24 scale sum |q_i k_i| (the
products' own roundings, their sum and the dequantisation), a weight by a
factor exp(2 e) from the scores of its key and of the maximum, and the
weighted mean of the values by that and the roundings of n weights:
    |O - exact| <= (2 (e^{2 e} - 1) + 64 * 2^-24) max |v|,
    |lse - exact| <= e + 64 * 2^-24 (1 + |lse|).
"""
import math

import numpy as np
import pytest
import torch

import hierarchical_routed_sparse_b200 as hga

import paged_ref as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
HELD = {"int8": hga.HGA_INT8, "e4m3": hga.HGA_E4M3}


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from hierarchical_routed_sparse_b200 import build
    build.build()
    hga.load()
    hga.device_check(clear=True)


def _params(B, Hq, Hkv, d, n_pages, chunks, dtype="bf16", cache="int8", k_c=-1, k_g=-1, scale=0.0):
    return hga.PagedParams(B, Hq, Hkv, d, n_pages, chunks, k_c, k_g,
                           hga.HGA_BF16 if dtype == "bf16" else hga.HGA_FP32, HELD[cache], scale)


def _cache(p, seed=0):
    """A cache whose pages are handed out in a shuffled order, everything in
    it filled so that a stray write or read shows."""
    g = torch.Generator().manual_seed(seed)
    c = hga.PagedCache(p)
    c.table.copy_(torch.randperm(p.n_pages, generator=g)[:p.B * p.max_chunks].view(p.B, p.max_chunks).int())
    for t in (c.k_pages, c.v_pages):
        t.view(torch.uint8).fill_(0x31)
    for t in (c.k_scale, c.v_scale, c.csum, c.gsum, c.k_tail, c.v_tail):
        t.fill_(float("nan"))
    return c


TENSORS = ("k_pages", "v_pages", "k_scale", "v_scale", "csum", "gsum", "k_tail", "v_tail")


def _bits(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def _snapshot(c):
    return {n: _bits(getattr(c, n)).copy() for n in TENSORS}


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _tokens(p, N, seed, layout="packed"):
    """q, k, v of N tokens as a projection leaves them."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(N, p.Hq + 2 * p.Hkv, p.d, generator=g).to(p.torch_dtype).cuda()
    if layout == "heads":                                       # [H][N][d] memory
        x = x.transpose(0, 1).contiguous().transpose(0, 1)
    return x[:, :p.Hq], x[:, p.Hq:p.Hq + p.Hkv], x[:, p.Hq + p.Hkv:]


class Plain:
    """What the cache should hold: every sequence's rotated keys and values."""

    def __init__(self, p, cache, table):
        self.p, self.kind, self.table = p, cache, table.cpu().numpy()
        self.k = [np.zeros((0, p.Hkv, p.d), np.float32) for _ in range(p.B)]
        self.v = [np.zeros((0, p.Hkv, p.d), np.float32) for _ in range(p.B)]

    def append(self, b, k, v, rope, inter):
        at = len(self.k[b])
        k = k.float().cpu().numpy()
        if rope is not None:
            k = R.rotate(k, rope.cpu().numpy()[at:at + len(k)][:, None], inter)
        self.k[b] = np.concatenate([self.k[b], k])
        self.v[b] = np.concatenate([self.v[b], v.float().cpu().numpy()])

    def check(self, c, before):
        """All of c: what was written, and that the rest is as before."""
        p = self.p
        now = _snapshot(c)
        want = {n: a.copy() for n, a in before.items()}
        el = 2 if p.dtype == hga.HGA_BF16 else 4
        csum, gsum = c.csum.cpu().numpy(), c.gsum.cpu().numpy()
        for b in range(p.B):
            n = len(self.k[b])
            for ch in range(n // 64):
                page = self.table[b, ch]
                rows = slice(64 * ch, 64 * ch + 64)
                for name, x in (("k", self.k[b][rows]), ("v", self.v[b][rows])):
                    x = x.transpose(1, 0, 2).reshape(p.Hkv * 8, 8, p.d)
                    code, scale = R.quantise(x, self.kind)
                    want[name + "_pages"][page] = code.reshape(p.Hkv, 64, p.d)
                    want[name + "_scale"][page] = scale.reshape(p.Hkv, 8).view(np.uint8)
                    if name == "k":
                        x = x.astype(np.float64).reshape(p.Hkv, 8, 8, p.d)
                        for got, axis in ((gsum[page], 2), (csum[page], (1, 2))):
                            tol = 64 * 2.0 ** -24 * np.abs(x).mean(axis)
                            assert (np.abs(got - x.mean(axis)) <= tol).all()
                want["csum"][page] = now["csum"][page]
                want["gsum"][page] = now["gsum"][page]
            if n:
                first = (n - 1) // 64 * 64
                kt = self.k[b][first:].transpose(1, 0, 2)
                vt = torch.from_numpy(np.ascontiguousarray(self.v[b][first:].transpose(1, 0, 2))).to(p.torch_dtype)
                want["k_tail"][b, :, :n - first] = np.ascontiguousarray(kt).view(np.uint8)
                want["v_tail"][b, :, :n - first] = vt.contiguous().view(torch.uint8).numpy().reshape(p.Hkv, n - first, p.d * el)
        for name in TENSORS:
            if name in ("k_tail", "v_tail"):                   # rows of earlier chunks may stay behind the open ones
                for b in range(p.B):
                    m = (len(self.k[b]) - 1) % 64 + 1 if len(self.k[b]) else 0
                    np.testing.assert_array_equal(now[name][b, :, :m], want[name][b, :, :m], err_msg=name)
                    if len(self.k[b]) <= 64:
                        np.testing.assert_array_equal(now[name][b, :, m:], before[name][b, :, m:], err_msg=name)
            else:
                np.testing.assert_array_equal(now[name], want[name], err_msg=name)


def _append(c, plain, lens, seed, rope, inter, layout="packed", pad=0, with_q=True, held=None):
    """One call: sequence b gets lens[b] tokens; returns q_out's check."""
    p = c.p
    N = sum(lens) + pad
    q, k, v = _tokens(p, N, seed, layout)
    have = [len(x) for x in plain.k] if held is None else held
    cu = np.concatenate([[0], np.cumsum(lens)])
    q_out = torch.full((N, p.Hq, p.d), 5.0, dtype=p.torch_dtype, device="cuda") if with_q else None
    c.append(_int32(have), k, v, cu=_int32(cu.tolist()), q=q if with_q else None, q_out=q_out, rope=rope, interleaved=inter)
    torch.cuda.synchronize()
    for b, n in enumerate(lens):
        if n:
            s = slice(cu[b], cu[b + 1])
            if with_q:
                x = q[s].float().cpu().numpy()
                t = np.zeros((n, 1, 0), np.float32) if rope is None else rope.cpu().numpy()[have[b]:have[b] + n][:, None]
                want = torch.from_numpy(R.rotate(x, t, inter)).to(p.torch_dtype)
                assert torch.equal(q_out[s].cpu(), want)
            plain.append(b, k[s], v[s], rope, inter)
    if with_q and pad:
        assert (q_out[cu[-1]:] == 5.0).all()                   # rows behind the last sequence


APPEND = [  # B, Hq, Hkv, d, dtype, cache, rot, interleaved, calls (tokens of each sequence)
    (1, 4, 1, 128, "bf16", "int8", 128, False, [[1], [62], [1], [64], [65]]),
    (3, 6, 2, 64, "fp32", "e4m3", 32, True, [[5, 0, 130], [60, 64, 1], [1, 63, 190]]),
    (2, 3, 3, 128, "fp32", "int8", 16, False, [[63, 127], [1, 1], [200, 3]]),
    (4, 8, 1, 64, "bf16", "e4m3", 64, False, [[64, 1, 0, 10], [0, 0, 0, 54], [1, 63, 300, 1]]),
    (2, 2, 1, 128, "bf16", "e4m3", 0, False, [[100, 28], [29, 100]]),
    (5, 5, 5, 64, "bf16", "int8", 48, True, [[1, 1, 1, 1, 1], [70, 63, 62, 64, 0], [1, 1, 1, 1, 1]]),
]


@pytest.mark.parametrize("layout", ["packed", "heads"])
@pytest.mark.parametrize("case", APPEND, ids=lambda c: "-".join(str(x) for x in c[:7]))
def test_append(case, layout):
    B, Hq, Hkv, d, dtype, kind, rot, inter, calls = case
    p = _params(B, Hq, Hkv, d, 8 * B + 2, 8, dtype, kind)
    c = _cache(p)
    plain, before = Plain(p, kind, c.table), _snapshot(c)
    rope = hga.rope_table(512, rot) if rot else None
    for i, lens in enumerate(calls):
        _append(c, plain, lens, 10 + i, rope, inter, layout, pad=3 * i, with_q=i != 1)
        plain.check(c, before)
    assert hga.device_check() == 0


def test_tokens_one_by_one_or_at_once():
    # 200 tokens in one call, in pieces, and one at a time without offsets.
    p = _params(1, 4, 2, 128, 5, 4, "bf16", "int8")
    rope = hga.rope_table(256, 128)
    q, k, v = _tokens(p, 200, 3)
    got = []
    for pieces in ([200], [1, 62, 1, 64, 22, 50], [1] * 200):
        c = _cache(p, seed=1)
        at = 0
        for n in pieces:
            cu = None if n == 1 else _int32([0, n])
            c.append(_int32([at]), k[at:at + n], v[at:at + n], cu=cu, rope=rope)
            at += n
        torch.cuda.synchronize()
        got.append(_snapshot(c))
        got[-1]["k_tail"], got[-1]["v_tail"] = got[-1]["k_tail"][:, :, :8], got[-1]["v_tail"][:, :, :8]
    for other in got[1:]:
        for n in TENSORS:
            np.testing.assert_array_equal(got[0][n], other[n], err_msg=n)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_groups_of_extremes(kind):
    # All zero, below the smallest scale, near the largest float, a NaN, an
    # infinity, and one large value among small ones.
    p = _params(1, 1, 1, 64, 3, 2, "fp32", kind)
    c = _cache(p)
    plain, before = Plain(p, kind, c.table), _snapshot(c)
    g = torch.Generator().manual_seed(2)
    x = torch.randn(64, 1, 64, generator=g)
    x[0:8] = 0
    x[8:16] *= 1e-41
    x[16:24] *= 5e37
    x[24, 0, 3] = float("nan")
    x[33, 0, 60] = float("-inf")
    x[40, 0, 0] = 1e20
    x = x.cuda()
    c.append(_int32([0]), x, x, cu=_int32([0, 64]))
    torch.cuda.synchronize()
    page = int(c.table[0, 0])
    for i in (3, 4):
        assert np.isnan(float(c.k_scale[page, 0, i])) and not c.k_pages[page, 0, 8 * i:8 * i + 8].view(torch.uint8).any()
    fine = [0, 1, 2, 5, 6, 7]
    code, scale = R.quantise(x.cpu().numpy()[:, 0].reshape(8, 8, 64)[fine], kind)
    np.testing.assert_array_equal(c.v_scale[page, 0].cpu().numpy()[fine], scale)
    np.testing.assert_array_equal(c.v_pages[page, 0].view(torch.uint8).cpu().numpy().reshape(8, 8, 64)[fine], code)
    assert plain.p is p and before["k_tail"].size


def test_faults_on_the_device_are_skipped_and_recorded():
    # Offsets outside the tokens, tokens past the table's width, a page that
    # is not in the pool, an empty slot: the other sequences are served and
    # nothing else is written.
    p = _params(6, 2, 1, 64, 30, 2, "bf16", "int8")
    c = _cache(p)
    c.table[4, 0] = 30
    c.table[5, 0] = -7
    plain, before = Plain(p, "int8", c.table), _snapshot(c)
    q, k, v = _tokens(p, 40, 1)
    #             served, offsets too far, decreasing, past the width, page, page
    pos = [0, 3, 0, 128, 60, 63]
    cu = [0, 10, 41, 12, 20, 26, 30]
    q_out = torch.full((40, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    hga.device_check(clear=True)
    checked = hga.checked_build()
    assert not checked
    c.append(_int32(pos), k, v, cu=_int32(cu), q=q, q_out=q_out)
    assert hga.device_check(clear=True) in (411, 412, 413)
    plain.append(0, k[:10], v[:10], None, False)
    now = _snapshot(c)
    for n in ("k_pages", "v_pages", "csum", "gsum", "k_scale", "v_scale"):
        np.testing.assert_array_equal(now[n], before[n], err_msg=n)
    np.testing.assert_array_equal(now["k_tail"][0, :, :10],
                                  np.ascontiguousarray(plain.k[0].transpose(1, 0, 2)).view(np.uint8))
    for b in (1, 2):
        np.testing.assert_array_equal(now["k_tail"][b], before["k_tail"][b])
    assert (q_out[12:20] == 5.0).all() and torch.equal(q_out[:10], q[:10])
    empty = _cache(p)
    was = _snapshot(empty)
    empty.append(_int32([-1] * 6), k, v, cu=_int32([0, 5, 10, 15, 20, 25, 30]), q=q, q_out=q_out.fill_(5.0))
    torch.cuda.synchronize()
    assert (q_out == 5.0).all() and all(np.array_equal(was[n], a) for n, a in _snapshot(empty).items())
    assert hga.device_check() == 0


# ---- decode ---------------------------------------------------------------------------

def _filled(p, kind, lens, seed=0, clustered=True):
    """A cache whose sequences hold lens[b] tokens (the queries' positions are
    lens[b] - 1): pages and open rows drawn directly, everything unused NaN
    or out of range."""
    g = torch.Generator().manual_seed(seed)
    c = _cache(p, seed)
    table = c.table.clone()
    c.table.fill_(p.n_pages + 1000)                            # chunks that are not complete: not read
    for b, n in enumerate(lens):
        closed = max(n - 1, 0) // 64
        for ch in range(closed):
            page = int(table[b, ch])
            c.table[b, ch] = page
            k = torch.randn(p.Hkv, 8, 8, p.d, generator=g)
            if clustered:
                k = 0.3 * k + torch.randn(p.Hkv, 1, 1, p.d, generator=g)
            v = torch.randn(p.Hkv, 8, 8, p.d, generator=g)
            c.csum[page] = k.mean((1, 2)).cuda()
            c.gsum[page] = k.mean(2).cuda()
            for name, x in (("k", k), ("v", v)):
                code, scale = R.quantise(x.view(-1, 8, p.d).numpy(), kind)
                getattr(c, name + "_pages").view(torch.uint8)[page] = torch.from_numpy(code).view(p.Hkv, 64, p.d).cuda()
                getattr(c, name + "_scale")[page] = torch.from_numpy(scale).view(p.Hkv, 8).cuda()
        rows = (n - 1) % 64 + 1 if n else 0
        c.k_tail[b, :, :rows] = torch.randn(p.Hkv, rows, p.d, generator=g).cuda()
        c.v_tail[b, :, :rows] = torch.randn(p.Hkv, rows, p.d, generator=g).to(p.torch_dtype).cuda()
    q = torch.randn(p.B, p.Hq, p.d, generator=g).to(p.torch_dtype).cuda()
    return c, q


def _decode(c, pos, q, rows=True):
    p = c.p
    wc, wg = hga.paged_widths(p)
    O = torch.full((p.B, p.Hq, p.d), 9.0, device="cuda")
    lse = torch.full((p.B, p.Hq), 9.0, device="cuda")
    cidx = torch.full((p.B, p.Hkv, wc), 9, dtype=torch.int32, device="cuda") if rows else None
    gidx = torch.full((p.B, p.Hkv, wg), 9, dtype=torch.int32, device="cuda") if rows else None
    c.decode(_int32(pos), q, O, lse, cidx, gidx)
    torch.cuda.synchronize()
    return O.cpu().numpy(), lse.cpu().numpy(), None if not rows else cidx.cpu().numpy(), None if not rows else gidx.cpu().numpy()


def _check_decode(c, kind, pos, q, got, rows=True):
    p = c.p
    O, lse, cidx, gidx = got
    G = p.Hq // p.Hkv
    scale = p.scale or 1.0 / math.sqrt(p.d)
    table = c.table.cpu().numpy()
    qs = q.double().cpu().numpy()
    codes = {n: getattr(c, n + "_pages").view(torch.uint8) for n in "kv"}
    for b in range(p.B):
        if pos[b] < 0:
            assert (O[b] == 0).all() and np.isneginf(lse[b]).all()
            if rows:
                assert (cidx[b] == -1).all() and (gidx[b] == -1).all()
            continue
        c0, open_rows = pos[b] // 64, pos[b] % 64 + 1
        pages = torch.from_numpy(table[b, :c0].astype(np.int64)).cuda()
        csum, gsum = c.csum[pages].double().cpu().numpy(), c.gsum[pages].double().cpu().numpy()
        kh, vh = (R.held(codes[n][pages].cpu().numpy().reshape(c0, p.Hkv, 8, 8, p.d),
                         getattr(c, n + "_scale")[pages].cpu().numpy(), kind) for n in "kv")
        kt, vt = c.k_tail[b, :, :open_rows].double().cpu().numpy(), c.v_tail[b, :, :open_rows].double().cpu().numpy()
        for h in range(p.Hkv):
            heads = slice(h * G, h * G + G)
            u = qs[b, heads].sum(0)
            chunks = R.top(csum[:, h] @ u, p.k_c if p.k_c > 0 else c0)
            ids = (8 * chunks[:, None] + np.arange(8)).reshape(-1)
            groups = ids[R.top(gsum[chunks, h].reshape(-1, p.d) @ u, p.k_g if p.k_g > 0 else len(ids))]
            if rows:
                for row, want in ((cidx[b, h], chunks), (gidx[b, h], groups)):
                    np.testing.assert_array_equal(row, np.concatenate([want, np.full(len(row) - len(want), -1)]))
            k = np.concatenate([kh[groups // 8, h, groups % 8].reshape(-1, p.d), kt[h]])
            v = np.concatenate([vh[groups // 8, h, groups % 8].reshape(-1, p.d), vt[h]])
            o_ref, l_ref = R.attend(qs[b, heads], k, v, scale)
            e = (p.d + 8) * 2.0 ** -24 * scale * (np.abs(qs[b, heads]) @ np.abs(k).T).max()
            tol = (2 * math.expm1(2 * e) + 64 * 2.0 ** -24) * np.abs(v).max()
            assert np.abs(O[b, heads] - o_ref).max() <= tol, (b, h, np.abs(O[b, heads] - o_ref).max(), tol)
            assert np.abs(lse[b, heads] - l_ref).max() <= e + 64 * 2.0 ** -24 * (1 + np.abs(l_ref).max())


DECODE = [  # Hq, Hkv, d, dtype, cache, k_c, k_g, lens
    (8, 2, 128, "bf16", "int8", 3, 13, [1, 64, 65, 700, 0, 128]),
    (4, 4, 64, "fp32", "e4m3", 2, 9, [333, 2, 640]),
    (16, 2, 128, "fp32", "int8", 4, 7, [449, 450]),
    (5, 1, 64, "bf16", "int8", 1, 1, [200, 129, 64, 63]),
    (6, 2, 128, "bf16", "e4m3", 5, 40, [577, 321, 0]),
    (7, 1, 128, "bf16", "e4m3", -1, 6, [640, 65]),
    (3, 1, 64, "fp32", "int8", 2, -1, [1, 500]),
    (4, 1, 128, "bf16", "int8", -1, -1, [640, 449, 0, 63]),
    (2, 2, 64, "bf16", "e4m3", -1, -1, [301]),
    (24, 3, 128, "fp32", "e4m3", -1, -1, [64, 192, 600]),
    (4, 2, 128, "bf16", "int8", 40, 100, [640, 100]),
]


@pytest.mark.parametrize("case", DECODE, ids=lambda c: "-".join(str(x) for x in c[:7]))
def test_decode(case):
    Hq, Hkv, d, dtype, kind, k_c, k_g, lens = case
    p = _params(len(lens), Hq, Hkv, d, 12 * len(lens), 11, dtype, kind, k_c, k_g)
    c, q = _filled(p, kind, lens)
    pos = [n - 1 for n in lens]
    _check_decode(c, kind, pos, q, _decode(c, pos, q))
    if k_c == k_g == -1:
        _check_decode(c, kind, pos, q, _decode(c, pos, q, rows=False), rows=False)
    assert hga.device_check() == 0


@pytest.mark.parametrize("k_c,k_g", [(8, 32), (16, 64), (-1, -1)])
@pytest.mark.parametrize("B,n,Hq,Hkv", [(1, 20001, 8, 2), (3, 5000, 4, 1), (40, 900, 16, 8)])
def test_decode_long_and_wide(B, n, Hq, Hkv, k_c, k_g):
    lens = [n] + [max(1, n - 61 * b) for b in range(1, B)]
    p = _params(B, Hq, Hkv, 128, sum(lens) // 64 + B, (n + 63) // 64, "bf16", "int8", k_c, k_g)
    c = _wide(p, lens)
    q = torch.randn(B, Hq, 128, device="cuda").bfloat16()
    pos = [m - 1 for m in lens]
    _check_decode(c, "int8", pos, q, _decode(c, pos, q, rows=k_c > 0), rows=k_c > 0)


def _wide(p, lens):
    """A filled cache made on the GPU (any codes, any summaries)."""
    c = hga.PagedCache(p)
    g = torch.Generator("cuda").manual_seed(4)
    c.k_pages.copy_(torch.randint(-127, 128, c.k_pages.shape, device="cuda", generator=g))
    c.v_pages.copy_(torch.randint(-127, 128, c.v_pages.shape, device="cuda", generator=g))
    for t in (c.k_scale, c.v_scale):
        t.uniform_(0.005, 0.03, generator=g)
    for t in (c.csum, c.gsum, c.k_tail):
        t.normal_(generator=g)
    c.v_tail.copy_(torch.randn(c.v_tail.shape, device="cuda", generator=g))
    at = 0
    order = torch.randperm(p.n_pages, device="cuda", generator=g).int()
    for b, n in enumerate(lens):
        m = (n + 63) // 64
        c.table[b, :m] = order[at:at + m]
        at += m
    return c


def test_equal_scores_go_to_the_lower_index():
    p = _params(1, 2, 1, 64, 12, 12, "fp32", "int8", 3, 5)
    c, q = _filled(p, "int8", [700])
    pages = c.table[0, :10].long()
    c.csum[pages[4:8]] = c.csum[pages[2]].clone()                       # five equal chunks
    c.gsum[pages[2:8]] = c.gsum[pages[2], :, :1].clone()                # whose groups are all equal
    u = q[0].double().sum(0)
    s = c.csum[pages, 0].double() @ u
    if float(s[2]) < float(s.median()):                          # make them the best
        q = -q
        s = -s
    c.csum[pages[[0, 1, 3, 8, 9]]] -= 100 * q[0].sum(0)
    got = _decode(c, [699], q)
    assert got[2][0, 0].tolist() == [2, 4, 5] and got[3][0, 0].tolist() == [16, 17, 18, 19, 20]
    _check_decode(c, "int8", [699], q, got)


def test_large_logits_and_uneven_values():
    # Scores in the hundreds; value groups 2^24 apart in size; tiny values.
    for kind in ("int8", "e4m3"):
        p = _params(2, 8, 1, 128, 22, 10, "fp32", kind)
        c, q = _filled(p, kind, [640, 300])
        q = 30 * q
        pages = c.table[0, :9].long()
        c.v_scale[pages[::2]] *= 2.0 ** 24
        c.v_scale[c.table[1, :4].long()] *= 2.0 ** -60
        c.v_tail[1] *= 2.0 ** -60
        for rows in (True, False):
            got = _decode(c, [639, 299], q, rows=rows)
            _check_decode(c, kind, [639, 299], q, got, rows=rows)


def test_scale_and_zero_values():
    p = _params(1, 4, 1, 64, 6, 6, "bf16", "int8", scale=0.5)
    c, q = _filled(p, "int8", [300])
    c.v_scale[c.table[0, :4].long()] = 2.0 ** -126               # groups that hold zeros
    c.v_pages[c.table[0, :4].long()] = 0
    c.v_tail.zero_()
    got = _decode(c, [299], q, rows=False)
    assert (got[0] == 0).all()
    _check_decode(c, "int8", [299], q, got, rows=False)


def test_a_held_nan_shows_only_where_it_is_attended():
    p = _params(2, 2, 2, 64, 20, 8, "bf16", "int8", 2, 4)
    c, q = _filled(p, "int8", [400, 400])
    clean = _decode(c, [399, 399], q)
    grp = int(clean[3][0, 1, 2])
    c.k_scale[int(c.table[0, grp // 8]), 1, grp % 8] = float("nan")
    got = _decode(c, [399, 399], q)
    assert np.isnan(got[0][0, 1]).all() and np.isnan(got[1][0, 1])
    keep = np.ones((2, 2), bool)
    keep[0, 1] = False
    np.testing.assert_array_equal(got[0][keep], clean[0][keep])
    np.testing.assert_array_equal(got[3], clean[3])


def test_bad_pages_and_positions_are_left_out():
    # A page outside the pool: its groups are left out (routed or dense); a
    # position past the table's width: an empty sequence.
    hga.device_check(clear=True)
    p = _params(2, 4, 1, 128, 20, 6, "bf16", "int8")
    c, q = _filled(p, "int8", [384, 100])
    keep = c.table.clone()
    c.table[0, 2] = 20
    O, lse, _, _ = _decode(c, [383, 384], q, rows=False)
    assert hga.device_check(clear=True) in (431, 432)
    assert (O[1] == 0).all() and np.isneginf(lse[1]).all()
    # what is left: chunks 0, 1, 3, 4 and the open rows
    k2 = _params(1, 4, 1, 128, 20, 5, "bf16", "int8")
    c2 = hga.PagedCache(k2, **{n: getattr(c, n)[:1].contiguous() if n in ("k_tail", "v_tail") else getattr(c, n) for n in TENSORS})
    c2.table[0, :4] = keep[0, [0, 1, 3, 4]]
    _check_decode(c2, "int8", [319], q[:1], (O[:1], lse[:1], None, None), rows=False)
    pr = _params(2, 4, 1, 128, 20, 6, "bf16", "int8", 2, 8)
    cr = hga.PagedCache(pr, **{n: getattr(c, n) for n in TENSORS + ("table",)})
    got = _decode(cr, [383, 99], q)
    assert hga.device_check(clear=True) == 421
    assert np.isfinite(got[0]).all() and 2 not in got[2][0, 0]


def test_shared_prefix_pages():
    p = _params(2, 4, 2, 128, 20, 8, "bf16", "int8", 3, 10)
    c, q = _filled(p, "int8", [400, 390])
    c.table[1, :5] = c.table[0, :5]
    _check_decode(c, "int8", [399, 389], q, _decode(c, [399, 389], q))


def test_offsets_past_32_bits():
    # Pages whose first byte, and whose summaries' first element, lie past 2^32.
    n = (1 << 32) // (64 * 128) // 2 + 40
    p = _params(1, 4, 2, 128, n, 10, "bf16", "int8", 2, 6)
    c = hga.PagedCache(p)
    far = torch.arange(n - 12, n, device="cuda")
    g = torch.Generator("cuda").manual_seed(1)
    c.table.copy_(far[torch.randperm(12, device="cuda", generator=g)[:10]].view(1, 10))
    assert n * 2 * 64 * 128 > 1 << 32
    rope = hga.rope_table(640, 128)
    q, k, v = _tokens(p, 600, 8)
    c.append(_int32([0]), k, v, cu=_int32([0, 600]), rope=rope)
    qn = torch.randn(1, 4, 128, device="cuda").bfloat16()
    got = _decode(c, [599], qn)
    plain = Plain(p, "int8", c.table)
    plain.append(0, k, v, rope, False)
    for ch in range(9):
        page = int(c.table[0, ch])
        x = plain.k[0][64 * ch:64 * ch + 64].transpose(1, 0, 2).reshape(16, 8, 128)
        code, scale = R.quantise(x, "int8")
        np.testing.assert_array_equal(c.k_pages[page].view(torch.uint8).cpu().numpy(), code.reshape(2, 64, 128))
        np.testing.assert_array_equal(c.k_scale[page].cpu().numpy(), scale.reshape(2, 8))
    assert not c.k_pages[:n - 12].any()
    _check_decode(c, "int8", [599], qn, got)


def test_two_streams_and_two_graphs_at_once():
    # Calls that overlap: one cache, workspaces of their own.
    p = _params(4, 8, 2, 128, 200, 40, "bf16", "int8")
    c, q = _filled(p, "int8", [2500, 1700, 64, 0])
    pos = _int32([2499, 1699, 63, -1])
    want = _decode(c, [2499, 1699, 63, -1], q, rows=False)
    ws = [torch.empty(hga.paged_workspace_size(p), dtype=torch.uint8, device="cuda") for _ in range(2)]
    O = [torch.empty(4, 8, 128, device="cuda") for _ in range(2)]
    lse = [torch.empty(4, 8, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs = []
    for i, s in enumerate(streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            c.decode(pos, q, O[i], lse[i], workspace=ws[i])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            c.decode(pos, q, O[i], lse[i], workspace=ws[i])
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for i in range(2):
        np.testing.assert_array_equal(O[i].cpu().numpy(), want[0])
        np.testing.assert_array_equal(lse[i].cpu().numpy(), want[1])


@pytest.mark.parametrize("dtype,kind,k_c,k_g", [("bf16", "int8", 2, 9), ("fp32", "e4m3", -1, -1)])
def test_generation_from_prompts(dtype, kind, k_c, k_g):
    # The operators together, as a program uses them: ragged prompts, then
    # tokens, the step captured once and replayed over chunk boundaries; every
    # step against the plain cache.
    B, Hq, Hkv, d, T = 3, 4, 2, 64, 400
    rope = hga.rope_table(T, d)
    st = hga.PagedDecodeState(B, Hq, Hkv, d, T, k_c, k_g, hga.HGA_BF16 if dtype == "bf16" else hga.HGA_FP32,
                              HELD[kind], rope=rope)
    p = st.p
    plain = Plain(p, kind, st.cache.table)
    lens = [100, 0, 260]
    _, k, v = _tokens(p, 360, 5)
    st.prefill(k, v, _int32([0, 100, 100, 360]))
    for b, s in ((0, slice(0, 100)), (2, slice(100, 360))):
        plain.append(b, k[s], v[s], rope, False)
    torch.cuda.synchronize()
    assert st.pos.tolist() == lens
    qkv = torch.zeros(B, Hq + 2 * Hkv, d, dtype=p.torch_dtype, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = None
    for step in range(90):
        x = torch.randn(qkv.shape, generator=torch.Generator().manual_seed(step)).to(p.torch_dtype)
        qkv.copy_(x)
        args = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        if step < 2:
            st.step(*args)
        else:
            if graph is None:
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    st.step(*args)
            graph.replay()
        torch.cuda.synchronize()
        for b in range(B):
            plain.append(b, x[b:b + 1, Hq:Hq + Hkv], x[b:b + 1, Hq + Hkv:], rope, False)
        pos = [len(plain.k[b]) - 1 for b in range(B)]
        assert st.pos.tolist() == [n + 1 for n in pos]
        rows = rope.cpu().numpy()[pos][:, None]
        turned = torch.from_numpy(R.rotate(x[:, :Hq].float().numpy(), rows, False)).to(p.torch_dtype)
        assert torch.equal(st.q.cpu(), turned)
        if step % 9 == 0 or any(n % 64 in (63, 0) for n in pos):
            got = (st.O.cpu().numpy(), st.lse.cpu().numpy()) + ((None, None) if st.gidx is None else
                                                               (st.cidx.cpu().numpy(), st.gidx.cpu().numpy()))
            _check_decode(st.cache, kind, pos, st.q, got, rows=st.gidx is not None)
    plain.check(st.cache, _snapshot(st.cache))
    assert hga.device_check() == 0 and hga.device_status() == 0


def test_append_many_sequences():
    # More sequences than lanes, most of them with a token or none, one with
    # several chunks (a thread counts the chunks of neighbouring sequences).
    B = 70
    p = _params(B, 4, 2, 64, 5 * B, 5, "bf16", "int8")
    c = _cache(p)
    plain, before = Plain(p, "int8", c.table), _snapshot(c)
    rope = hga.rope_table(320, 64)
    rng = np.random.default_rng(3)
    for i in range(3):
        lens = rng.integers(0, 3, B).tolist()
        lens[int(rng.integers(B))] = [170, 64, 40][i]
        _append(c, plain, lens, 40 + i, rope, False, pad=2)
    plain.check(c, before)
    # All of them at a chunk's last token, one token each, without offsets.
    for b in range(B):
        have = len(plain.k[b])
        if have % 64 != 63:
            n = 63 - have % 64
            _append(c, plain, [n if x == b else 0 for x in range(B)], 100 + b, rope, False, with_q=False)
    q, k, v = _tokens(p, B, 7)
    have = [len(x) for x in plain.k]
    c.append(_int32(have), k, v, rope=rope)
    torch.cuda.synchronize()
    for b in range(B):
        plain.append(b, k[b:b + 1], v[b:b + 1], rope, False)
    plain.check(c, before)
    assert hga.device_check() == 0


@pytest.mark.parametrize("n,k_c,k_g", [(60000, 8, 32), (60000, 33, 300), (60000, 200, 700), (60000, -1, 40),
                                       (140000, 16, 64), (140000, -1, -1)])
def test_many_chunks(n, k_c, k_g):
    # Selections of more keys than a warp holds (thinned, or bisected in shared
    # memory), tables past the part that is staged.
    p = _params(2, 4, 1, 64, n // 64 + 40, n // 64 + 20, "bf16", "e4m3", k_c, k_g)
    c = hga.PagedCache(p)
    g = torch.Generator("cuda").manual_seed(6)
    for t in (c.k_pages, c.v_pages):
        t.copy_((torch.randn(t.shape, device="cuda", generator=g) * 60).clamp(-400, 400).to(torch.float8_e4m3fn))
    for t in (c.k_scale, c.v_scale):
        t.uniform_(0.003, 0.01, generator=g)
    for t in (c.csum, c.gsum, c.k_tail):
        t.normal_(generator=g)
    c.v_tail.copy_(torch.randn(c.v_tail.shape, device="cuda", generator=g))
    order = torch.randperm(p.n_pages, device="cuda", generator=g).int()
    c.table[0, :n // 64] = order[:n // 64]
    c.table[1, :30] = order[-30:]
    q = torch.randn(2, 4, 64, device="cuda", generator=g).bfloat16()
    pos = [n - 1, 1900]
    rows = k_c > 0 or k_g > 0
    _check_decode(c, "e4m3", pos, q, _decode(c, pos, q, rows=rows), rows=rows)


@pytest.mark.parametrize("size", [1e33, 1e-30])
def test_queries_of_extreme_size(size):
    # Scores so far apart that one key takes all the weight, or so near zero
    # that all keys weigh the same: 2^-20 allows for a weight's two parts, its
    # exponential and the sums.
    p = _params(1, 8, 1, 128, 12, 10, "fp32", "int8")
    c, q = _filled(p, "int8", [600])
    q = q * size
    O, lse, _, _ = _decode(c, [599], q, rows=False)
    pages = c.table[0, :9].long()
    u8 = lambda t: t[pages].view(torch.uint8).cpu().numpy().reshape(9, 8, 8, 128)  # noqa: E731
    k = R.held(u8(c.k_pages), c.k_scale[pages, 0].cpu().numpy(), "int8").reshape(-1, 128)
    v = R.held(u8(c.v_pages), c.v_scale[pages, 0].cpu().numpy(), "int8").reshape(-1, 128)
    k = np.concatenate([k, c.k_tail[0, 0, :24].double().cpu().numpy()])
    v = np.concatenate([v, c.v_tail[0, 0, :24].double().cpu().numpy()])
    o_ref, l_ref = R.attend(q[0].double().cpu().numpy(), k, v, 1 / math.sqrt(128))
    assert np.abs(O[0] - o_ref).max() <= 2.0 ** -20 * np.abs(v).max()
    assert (np.abs(lse[0] - l_ref) <= 2.0 ** -20 * (1 + np.abs(l_ref))).all()


@pytest.mark.parametrize("long_at", [0, 17, 39])
def test_dense_batch_of_uneven_lengths(long_at):
    # One long sequence, cut over most of the GPU, among short and empty ones
    # that stay whole.
    lens = [1 + 37 * b % 300 for b in range(40)]
    lens[5] = lens[20] = 0
    lens[long_at] = 20011
    p = _params(40, 8, 2, 128, sum(n // 64 + 1 for n in lens), 313, "bf16", "int8")
    c = _wide(p, lens)
    q = torch.randn(40, 8, 128, device="cuda").bfloat16()
    pos = [n - 1 for n in lens]
    _check_decode(c, "int8", pos, q, _decode(c, pos, q, rows=False), rows=False)


@pytest.mark.parametrize("B,Hkv,n", [(33, 3, 64), (1, 1, 65), (2, 1, 700), (7, 5, 257), (100, 2, 1), (13, 1, 4000)])
def test_dense_borders(B, Hkv, n):
    # Units around the sizes at which a CTA's share begins and ends in them.
    lens = [max(1, n - 61 * (b % 5)) for b in range(B)]
    p = _params(B, 2 * Hkv, Hkv, 64, B * (n // 64 + 1), n // 64 + 1, "fp32", "e4m3")
    c, q = _filled(p, "e4m3", lens, clustered=False)
    pos = [m - 1 for m in lens]
    _check_decode(c, "e4m3", pos, q, _decode(c, pos, q, rows=False), rows=False)
    assert hga.device_check() == 0


@pytest.mark.parametrize("d,dtype,kind", [(128, "bf16", "int8"), (64, "fp32", "e4m3"), (128, "fp32", "int8"), (64, "bf16", "e4m3")])
@pytest.mark.parametrize("B,Hkv,width", [(100, 3, 6), (100, 3, 250), (100, 3, 900), (100, 3, 1100), (100, 3, 2100),  # four CTAs an SM
                                         (50, 4, 250), (50, 4, 1100),                         # two
                                         (25, 4, 250), (25, 4, 1100), (6, 8, 1100)])          # one, clusters
def test_every_split(B, Hkv, width, d, dtype, kind):
    # The warps and CTAs that a unit gets and the room for open rows follow from
    # the number of units and the table's width; lengths of every count of open tiles.
    lens = [(1 + 37 * b) % 330 for b in range(B)]
    lens[3] = 0
    lens[B - 1] = 320
    G = 1 + (width + B) % 8
    p = _params(B, Hkv * G, Hkv, d, sum(n // 64 + 1 for n in lens), width, dtype, kind, 3, 11)
    c, q = _short_tables(p, kind, lens)
    pos = [n - 1 for n in lens]
    _check_decode(c, kind, pos, q, _decode(c, pos, q))
    assert hga.device_check() == 0


def _short_tables(p, kind, lens):
    """A filled cache whose tables are far wider than the sequences are long."""
    narrow = _params(p.B, p.Hq, p.Hkv, p.d, p.B * 6, 6, "bf16" if p.dtype == hga.HGA_BF16 else "fp32", kind, 3, 11)
    made, q = _filled(narrow, kind, lens)
    c = hga.PagedCache(hga.PagedParams(p.B, p.Hq, p.Hkv, p.d, p.B * 6, p.max_chunks, p.k_c, p.k_g, p.dtype, p.cache_dtype),
                       **{n: getattr(made, n) for n in TENSORS})
    c.table[:, :min(6, p.max_chunks)] = made.table[:, :min(6, p.max_chunks)]
    return c, q


@pytest.mark.parametrize("n_chunks,k_c,k_g", [(100, 8, 13), (200, 8, 20), (400, 8, 32), (400, 20, 32), (700, 8, 32), (700, 30, 40)])
@pytest.mark.parametrize("near", [2, 11, 25])
def test_scores_that_differ_in_their_last_bits(n_chunks, k_c, k_g, near):
    # The highest scores are 1 + j 2^-40 (two of each j): float64 tells them
    # apart, its first 32 bits do not.
    p = _params(1, 1, 1, 64, n_chunks + 1, n_chunks + 1, "fp32", "int8", k_c, k_g)
    lens = [64 * n_chunks + 7]
    c = _wide(p, lens)
    g = torch.Generator().manual_seed(near)
    pages = c.table[0, :n_chunks].long()
    for t, n in ((c.csum, n_chunks), (c.gsum, 8 * n_chunks)):
        s = torch.zeros(n, 64)
        s[:, 0] = torch.rand(n, generator=g) * 0.9
        top = torch.randperm(n, generator=g)[:near]
        s[top, 0] = 1.0
        s[top, 1] = torch.arange(near).div(2, rounding_mode="floor").float() * 2.0 ** -40
        t[pages] = s.view(n_chunks, *t.shape[1:]).cuda()
    q = torch.zeros(1, 1, 64, device="cuda")
    q[..., :2] = 1.0
    _check_decode(c, "int8", [lens[0] - 1], q, _decode(c, [lens[0] - 1], q))
