"""The generation loop (PagedDecodeState): empty and held slots, and its limits."""
import numpy as np
import pytest
import torch

import hierarchical_routed_sparse_b200 as hga

import paged_ref as R
from test_gpu_paged import Plain, _check_decode, _int32, _tokens

pytestmark = pytest.mark.gpu
FORMS = [("bf16", "int8", 2, 9), ("fp32", "e4m3", -1, -1)]


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from hierarchical_routed_sparse_b200 import build
    build.build()
    hga.load()
    hga.device_check(clear=True)


def _state(B, T, dtype, kind, k_c, k_g, rope, **kw):
    return hga.PagedDecodeState(B, 4, 2, 64, T, k_c, k_g, hga.HGA_BF16 if dtype == "bf16" else hga.HGA_FP32,
                                hga.HGA_INT8 if kind == "int8" else hga.HGA_E4M3, rope=rope, **kw)


def _token(st, seed):
    x = torch.randn(st.p.B, 8, 64, generator=torch.Generator().manual_seed(seed)).to(st.p.torch_dtype).cuda()
    return x[:, :4], x[:, 4:6], x[:, 6:]


def _check_step(st, kind, plain, rope, seed, live):
    """The step of token `seed` that has just run, for the sequences in `live`;
    the others are answered as empty."""
    q, k, v = _token(st, seed)
    torch.cuda.synchronize()
    pos = [-1] * st.p.B
    for b in live:
        plain.append(b, k[b:b + 1], v[b:b + 1], rope, False)
        pos[b] = len(plain.k[b]) - 1
        x = q[b:b + 1].float().cpu().numpy()
        if rope is not None:
            x = R.rotate(x, rope.cpu().numpy()[pos[b]][None, None], False)
        assert torch.equal(st.q[b:b + 1].cpu(), torch.from_numpy(x).to(st.p.torch_dtype))
    rows = st.gidx is not None
    got = (st.O.cpu().numpy(), st.lse.cpu().numpy()) + ((st.cidx.cpu().numpy(), st.gidx.cpu().numpy()) if rows else (None, None))
    _check_decode(st.cache, kind, pos, st.q, got, rows=rows)


def _captured(st, seeds):
    """Steps of the tokens `seeds`: one to warm up, then replays of a graph;
    yields after each."""
    qkv = [t.clone() for t in _token(st, 0)]
    graph = None
    for i, seed in enumerate(seeds):
        for t, x in zip(qkv, _token(st, seed)):
            t.copy_(x)
        if i == 0:
            st.step(*qkv)
        else:
            if graph is None:
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    st.step(*qkv)
            graph.replay()
        yield seed


@pytest.mark.parametrize("dtype,kind,k_c,k_g", FORMS)
def test_an_empty_slot_stays_empty(dtype, kind, k_c, k_g):
    # A slot at -1 through a prefill that has tokens for it and through captured
    # steps over a chunk's end: it is not counted, not written and answered as empty.
    rope = hga.rope_table(256, 64)
    st = _state(3, 256, dtype, kind, k_c, k_g, rope)
    plain = Plain(st.p, kind, st.cache.table)
    st.pos[1] = -1
    _, k, v = _tokens(st.p, 95, 5)
    st.prefill(k, v, _int32([0, 70, 90, 95]))
    for b, s in ((0, slice(0, 70)), (2, slice(90, 95))):
        plain.append(b, k[s], v[s], rope, False)
    torch.cuda.synchronize()
    assert st.pos.tolist() == [70, -1, 5]
    for i, seed in enumerate(_captured(st, range(64))):
        _check_step(st, kind, plain, rope, seed, (0, 2))
        assert st.pos.tolist() == [71 + i, -1, 6 + i]
    c = st.cache
    pages = c.table[1].long()
    assert not c.k_tail[1].any() and not c.v_tail[1].any()
    for t in (c.k_pages, c.v_pages, c.k_scale, c.v_scale, c.csum, c.gsum):
        assert not t[pages].view(torch.uint8).any()
    assert hga.device_check() == 0


def test_a_held_sequence_goes_on_where_it_was():
    # Sequence 1 is held (its position set aside, -1 in its place) for four steps
    # of the others: what it then generates is what it generates without them.
    rope = hga.rope_table(192, 64)
    outs = []
    for hold in (False, True):
        st = _state(2, 192, "bf16", "int8", 2, 9, rope)
        _, k, v = _tokens(st.p, 130, 6)
        st.prefill(k, v, _int32([0, 10, 130]))
        got = []
        for step in range(12):
            if hold and step == 5:
                kept = st.pos[1].clone()
                st.pos[1] = -1
                for extra in range(4):
                    O = st.step(*_token(st, 100 + extra))
                    assert (O[1] == 0).all() and st.pos.tolist()[1] == -1
                st.pos[1] = kept
            got.append(st.step(*_token(st, step))[1].clone())
        assert st.pos.tolist() == [26 if hold else 22, 132]
        outs.append(torch.stack(got))
    assert torch.equal(*outs)


def test_positions_move_by_the_tokens_taken():
    # Each against what append writes: an empty slot, offsets that are not taken,
    # tokens past the rotation table's end, past the cache's, none at all.
    p = hga.PagedParams(7, 2, 1, 64, 14, 2)
    c = hga.PagedCache(p, table=torch.arange(14, dtype=torch.int32, device="cuda").view(7, 2))
    g = torch.Generator().manual_seed(2)
    k = torch.randn(60, 1, 64, generator=g).bfloat16().cuda()
    cu = _int32([0, 10, 20, 71, 30, 40, 40, 60])
    pos, rope = _int32([5, -3, 0, 90, 95, 128, 0]), hga.rope_table(100, 64)
    for tab, want in ((rope, [15, -3, 0, 90, 100, 128, 20]), (None, [15, -3, 0, 90, 105, 128, 20])):
        now, last = pos.clone(), _int32([9] * 7)
        hga.device_check(clear=True)
        c.advance(now, cu=cu, N=60, rope=tab, last=last)
        assert now.tolist() == want
        assert last.tolist() == [14, -1, -1, -1, want[4] - 1, -1, 19]
        assert hga.device_check(clear=True) in (412, 413)
        for t in (c.k_tail, c.v_tail):
            t.fill_(7.0)
        c.append(pos, k, k, cu=cu, rope=tab)
        assert hga.device_check(clear=True) in (412, 413)
        rows = [int((c.k_tail[b, 0] != 7.0).any(1).sum()) for b in range(7)]
        assert rows == [10, 0, 0, 0, want[4] - 95, 0, 20]
    one = _int32([5, -3, 0, 90, 95, 128, 127])
    c.advance(one)
    assert one.tolist() == [6, -3, 1, 91, 96, 128, 128]
    assert hga.device_check(clear=True) == 413
    with pytest.raises(ValueError):
        c.advance(one, cu=cu)
    many = hga.PagedParams(600, 2, 1, 64, 600, 1)
    cm = hga.PagedCache(many)
    pos = torch.arange(-300, 300, dtype=torch.int32, device="cuda") % 64 - 2
    want = torch.where(pos < 0, pos, pos + 1)
    cm.advance(pos)
    assert torch.equal(pos, want) and hga.device_check() == 0


@pytest.mark.parametrize("dtype,kind,k_c,k_g", FORMS)
def test_a_full_sequence_does_not_count_on(dtype, kind, k_c, k_g):
    # Captured steps past the cache's end, and a prompt that does not fit: `pos`
    # stays at the end, the fault is recorded, O is 0, the others go on.
    st = _state(2, 128, dtype, kind, k_c, k_g, None)
    plain = Plain(st.p, kind, st.cache.table)
    _, k, v = _tokens(st.p, 130, 8)
    st.prefill(k, v, _int32([0, 126, 130]))
    for b, s in ((0, slice(0, 126)), (1, slice(126, 130))):
        plain.append(b, k[s], v[s], None, False)
    assert hga.device_check(clear=True) == 0
    for i, seed in enumerate(_captured(st, range(6))):
        _check_step(st, kind, plain, None, seed, (0, 1) if i < 2 else (1,))
        assert st.pos.tolist() == [min(127 + i, 128), 5 + i]
        assert (hga.device_check(clear=True) != 0) == (i >= 2)
    st.prefill(k, v, _int32([0, 0, 130]))
    assert st.pos.tolist() == [128, 128]
    assert hga.device_check(clear=True) == 413


@pytest.mark.parametrize("dtype,kind,k_c,k_g", FORMS)
@pytest.mark.parametrize("rows", [100, 127])
def test_a_rotation_table_that_ends_inside_the_last_chunk(rows, dtype, kind, k_c, k_g):
    # The table ends before the pages do: past its last row a token is not taken
    # and nothing is answered from what is left of the step before.
    rope = hga.rope_table(rows, 64)
    st = _state(2, 100, dtype, kind, k_c, k_g, rope)
    assert st.capacity == rows
    plain = Plain(st.p, kind, st.cache.table)
    _, k, v = _tokens(st.p, rows + 2, 9)
    st.prefill(k, v, _int32([0, rows - 2, rows + 2]))
    for b, s in ((0, slice(0, rows - 2)), (1, slice(rows - 2, rows + 2))):
        plain.append(b, k[s], v[s], rope, False)
    assert hga.device_check(clear=True) == 0
    for i, seed in enumerate(_captured(st, range(6))):
        _check_step(st, kind, plain, rope, seed, (0, 1) if i < 2 else (1,))
        assert st.pos.tolist() == [min(rows - 1 + i, rows), 5 + i]
        assert hga.device_check(clear=True) == (413 if i >= 2 else 0)


def test_limits_that_the_host_knows():
    with pytest.raises(ValueError, match="shorter"):
        _state(1, 129, "bf16", "int8", 2, 9, hga.rope_table(128, 64))
    st = _state(2, 100, "bf16", "int8", 2, 9, None)
    assert st.capacity == 128
    _, k, v = _tokens(st.p, 300, 1)                             # behind the offsets: tokens of no sequence
    st.prefill(k, v, _int32([0, 100, 120]))
    assert st.pos.tolist() == [100, 20] and hga.device_check() == 0
    with pytest.raises(ValueError):
        _state(1, 0, "bf16", "int8", 2, 9, None)
