"""Cases of the paged 8-bit key / value cache and the position rotation: their
inputs, their plain forms in elementary torch operations, their definitions in
64 bits, and the calls a user makes of them.

append  tokens of a ragged batch join the cache: queries and keys are rotated,
        open chunks keep their rows exactly, complete 64-token chunks are held
        in 8 bits with a scale for each 8-token group and kv-head, beside their
        chunk and group summaries
decode  one query per sequence attends the routed groups of its cache, or all
        of it (k_c = k_g = -1), and its open chunk
rope    the rotation between the projections' layout and the attention's, and
        its gradient
"""
import math
import random

import torch

own = False

CHUNK, GROUP = 64, 8
TINY = 2.0 ** -126                     # smallest normal float32
LEVEL = {"int8": 127.0, "e4m3": 448.0}
TORCH = {"bf16": torch.bfloat16, "fp32": torch.float32, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "fp32": 4}


# ---- the cases -----------------------------------------------------------------------

def listed():
    return [
        # One stream of generation: the next token of one sequence (32 q-heads, 8 kv-heads, d 128). Latency.
        dict(name="append, 1 stream", op="append", B=1, tokens=1, start=9000, Hq=32, Hkv=8, d=128, dtype="bf16",
             cache="int8", rot=128, interleaved=False, lay=1),
        # A batch of 64 streams at positions of their own, one token each; some complete a chunk.
        dict(name="append, 64 streams", op="append", B=64, tokens=1, start=2000, Hq=32, Hkv=8, d=128, dtype="bf16",
             cache="int8", rot=128, interleaved=False, lay=2),
        # Ragged prompts that go on from the middle of a chunk; float32, small heads, half of each head rotated.
        dict(name="append, ragged fp32", op="append", B=7, tokens=1500, start=300, Hq=6, Hkv=2, d=64, dtype="fp32",
             cache="e4m3", rot=32, interleaved=True, lay=3),
        # A long prompt in one call.
        dict(name="append, 16K prompt", op="append", B=1, tokens=16384, start=0, Hq=32, Hkv=8, d=128, dtype="bf16",
             cache="e4m3", rot=128, interleaved=False, lay=4),
        # The first tokens of a small model: less than two chunks, nothing to choose from.
        dict(name="decode, first tokens", op="decode", B=2, ctx=100, Hq=4, Hkv=2, d=64, dtype="fp32", cache="int8",
             k_c=2, k_g=9, lay=5),
        # One stream at 16K context: the generation step of the repository's benchmark, from an 8-bit cache.
        dict(name="decode, 1 x 16K", op="decode", B=1, ctx=16384, Hq=32, Hkv=8, d=128, dtype="bf16", cache="int8",
             k_c=8, k_g=32, lay=6),
        # A serving batch at up to 16K, positions of their own, one slot empty.
        dict(name="decode, 64 x 16K", op="decode", B=64, ctx=16384, Hq=32, Hkv=8, d=128, dtype="bf16", cache="int8",
             k_c=8, k_g=32, lay=7),
        # Long contexts with a larger routing budget.
        dict(name="decode, 4 x 128K", op="decode", B=4, ctx=131072, Hq=32, Hkv=8, d=128, dtype="bf16", cache="e4m3",
             k_c=16, k_g=64, lay=8),
        # Dense attention over the whole 8-bit cache of a batch: the yardstick that routing is compared with.
        dict(name="decode, all of 8 x 16K", op="decode", B=8, ctx=16384, Hq=32, Hkv=8, d=128, dtype="bf16",
             cache="int8", k_c=-1, k_g=-1, lay=9),
        # Dense attention of one long stream: few rows, a long axis.
        dict(name="decode, all of 1 x 50K", op="decode", B=1, ctx=50001, Hq=8, Hkv=2, d=128, dtype="bf16",
             cache="e4m3", k_c=-1, k_g=-1, lay=10),
        # A training segment's queries: projections (float32) to the attention's layout and type.
        dict(name="rope, segment", op="rope", B=1, T=2048, H=32, d=128, src="fp32", dst="bf16", rot=128, pos0=14336,
             interleaved=False, back=False),
        # The gradient for a batch of long segments, from the attention's float32 to the projections' type.
        dict(name="rope, gradient 4 x 4K", op="rope", B=4, T=4096, H=32, d=128, src="fp32", dst="bf16", rot=128,
             pos0=0, interleaved=False, back=True),
    ]


def _log(rng, lo, hi):
    """A whole number of lo..hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "append", "decode", "decode", "decode", "rope"])
    d = rng.choice([64, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    cache = rng.choice(["int8", "e4m3"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    Hq = Hkv * rng.randint(1, 8)
    rot = rng.choice([d, d, d // 2, d // 4])
    inter = rng.random() < 0.4
    lay = rng.randrange(1 << 30)
    if op == "append":
        B = _log(rng, 1, 64)
        tokens = 1 if rng.random() < 0.4 else _log(rng, 1, 6000 // B)
        return dict(op=op, B=B, tokens=tokens, start=_log(rng, 1, 2000), Hq=Hq, Hkv=Hkv, d=d, dtype=dtype,
                    cache=cache, rot=rot, interleaved=inter, lay=lay)
    if op == "decode":
        B = _log(rng, 1, 64)
        k_c, k_g = rng.randint(1, 16), rng.randint(1, 64)
        most = (1 << 19) // B
        if rng.random() < 0.35:
            k_c = k_g = -1
            most = (1 << 16) // B
        return dict(op=op, B=B, ctx=_log(rng, 1, min(131072, most)), Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, cache=cache,
                    k_c=k_c, k_g=k_g, lay=lay)
    T, H = _log(rng, 1, 4096), _log(rng, 1, 32)
    return dict(op=op, B=rng.randint(1, 4), T=T, H=H, d=d, src=dtype, dst=rng.choice(["bf16", "fp32"]), rot=rot,
                pos0=_log(rng, 1, 100000), interleaved=inter, back=rng.random() < 0.5)


def _layout(case):
    """Positions and token counts of a case's sequences, the same for every seed."""
    r = random.Random(case["lay"])
    B = case["B"]
    if case["op"] == "decode":
        pos = [case["ctx"] - 1] + [r.randint(case["ctx"] // 4, case["ctx"] - 1) for _ in range(B - 1)]
        if B >= 4:
            pos[2] = -1                                       # an empty slot of the batch
        return pos, [1] * B
    n = [case["tokens"]] + [r.randint(1, case["tokens"]) for _ in range(B - 1)]
    pos = [case["start"]] + [r.randint(0, case["start"]) for _ in range(B - 1)]
    for b in range(3, B, 8):                                  # some streams fill their chunk with this call
        pos[b] += -(pos[b] + n[b]) % CHUNK
    return pos, n


def _chunks(case):
    """Chunks that append touches: (first, how many) of each sequence, and how many of them it completes."""
    pos, n = _layout(case)
    first = [p // CHUNK for p in pos]
    count = [(p + m - 1) // CHUNK - p // CHUNK + 1 for p, m in zip(pos, n)]
    closed = sum((p + m) // CHUNK - p // CHUNK for p, m in zip(pos, n))
    return first, count, closed


def work(case):
    d = case["d"]
    if case["op"] == "rope":
        n = case["B"] * case["T"] * case["H"] * d
        table = case["T"] * case["rot"] * 4
        return dict(bytes=n * (SIZE[case["src"]] + SIZE[case["dst"]]) + table,
                    flops=3.0 * n * case["rot"] / d)
    Hq, Hkv, el, B = case["Hq"], case["Hkv"], SIZE[case["dtype"]], case["B"]
    pos, n = _layout(case)
    page = Hkv * (2 * CHUNK * d + 2 * GROUP * 4 + (1 + CHUNK // GROUP) * d * 4)   # codes, scales, summaries
    row = Hkv * d * (4 + el)                                                    # a row of the open chunk
    if case["op"] == "append":
        N = sum(n)
        kept = sum(min(m, (p + m - 1) % CHUNK + 1) for p, m in zip(pos, n))       # rows the open chunks get
        joined = sum(p % CHUNK for p, m in zip(pos, n) if p % CHUNK + m >= CHUNK)  # rows closed with the new ones
        closed = _chunks(case)[2]
        return dict(bytes=2 * N * Hq * d * el + 2 * N * Hkv * d * el + N * case["rot"] * 4 + (kept + joined) * row
                    + closed * page + closed * 4 + 4 * (2 * B + 1),
                    flops=3.0 * N * (Hq + Hkv) * case["rot"] + closed * Hkv * CHUNK * d * 8.0)
    G = Hq // Hkv
    nbytes = B * Hq * (d * el + d * 4 + 4) + 4 * B
    flops = 0.0
    for p in pos:
        if p < 0:
            continue
        c0, own_rows = p // CHUNK, p % CHUNK + 1
        nbytes += own_rows * row + 4 * c0
        k_c, k_g = case["k_c"], case["k_g"]
        n_c = c0 if k_c < 0 else min(k_c, c0)
        n_g = 8 * n_c if k_g < 0 else min(k_g, 8 * n_c)
        nbytes += Hkv * n_g * (2 * GROUP * d + 8)
        if k_c >= 0:
            nbytes += Hkv * (4 * k_c + (c0 * d * 4 if k_c < c0 else 0))
            flops += 2.0 * Hkv * c0 * d
        if k_g >= 0:
            nbytes += Hkv * (4 * k_g + (8 * n_c * d * 4 if k_g < 8 * n_c else 0))
            flops += 2.0 * Hkv * 8 * n_c * d
        flops += 4.0 * Hkv * G * d * (n_g * GROUP + own_rows)
    return dict(bytes=nbytes, flops=flops)


# ---- inputs ----------------------------------------------------------------------------

def _table(rows, rot):
    """cos | sin of the positions' angles (base 10000), formed in 64 bits."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(rows, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float().cuda()


def _quantise(x, cache):
    """Codes and scales of x [..., 8, d]: one scale for each group."""
    top = LEVEL[cache]
    a = x.abs().amax((-2, -1))
    safe = a.clamp(min=top * TINY)
    fine = torch.isfinite(a)
    y = x * (top / safe)[..., None, None]
    y = torch.where(fine[..., None, None], y, torch.zeros_like(y))
    code = y.round().to(torch.int8) if cache == "int8" else y.to(torch.float8_e4m3fn)
    return code, torch.where(fine, safe / top, torch.full_like(a, float("nan")))


def _pages(n, case, gen, cent=None):
    """The pages of a cache: random keys (around a centre for each page) and values, held as the cache holds them."""
    Hkv, d, dev = case["Hkv"], case["d"], "cuda"
    kind = TORCH[case["cache"]]
    s = dict(k_pages=torch.empty(n, Hkv, CHUNK, d, dtype=kind, device=dev),
             v_pages=torch.empty(n, Hkv, CHUNK, d, dtype=kind, device=dev),
             k_scale=torch.empty(n, Hkv, 8, device=dev), v_scale=torch.empty(n, Hkv, 8, device=dev),
             csum=torch.empty(n, Hkv, d, device=dev), gsum=torch.empty(n, Hkv, 8, d, device=dev))
    step = max(1, (1 << 26) // (Hkv * CHUNK * d))
    for a in range(0, n, step):
        m = min(step, n - a)
        k = torch.randn(m, Hkv, 8, 8, d, device=dev, generator=gen)
        if cent is not None:
            k = 0.3 * k + cent[a:a + m, :, None, None, :]
        v = torch.randn(m, Hkv, 8, 8, d, device=dev, generator=gen)
        for x, name in ((k, "k"), (v, "v")):
            code, scale = _quantise(x, case["cache"])
            s[name + "_pages"][a:a + m] = code.view(m, Hkv, CHUNK, d)
            s[name + "_scale"][a:a + m] = scale
        s["csum"][a:a + m] = k.mean((2, 3))
        s["gsum"][a:a + m] = k.mean(3)
    return s


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    randn = lambda *shape: torch.randn(*shape, device="cuda", generator=gen)  # noqa: E731
    if case["op"] == "rope":
        B, T, H, d = case["B"], case["T"], case["H"], case["d"]
        shape = (B, H, T, d) if case["back"] else (B, T, H, d)
        to = (B, T, H, d) if case["back"] else (B, H, T, d)
        return dict(case=case, x=randn(*shape).to(TORCH[case["src"]]), table=_table(case["pos0"] + T, case["rot"]),
                    y=torch.zeros(to, dtype=TORCH[case["dst"]], device="cuda"))
    B, Hq, Hkv, d, dt = case["B"], case["Hq"], case["Hkv"], case["d"], TORCH[case["dtype"]]
    pos, n = _layout(case)
    width = max((p + m - 1) // CHUNK + 1 for p, m in zip(pos, n))
    pages = [0 if p < 0 else (p + m - 1) // CHUNK + 1 for p, m in zip(pos, n)]
    total = sum(pages)
    spare = torch.randperm(total + 3, device="cuda", generator=gen)[:total].int()   # pages as an allocator leaves them
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    slot = torch.tensor([b * width + c for b in range(B) for c in range(pages[b])], dtype=torch.int64, device="cuda")
    table.view(-1)[slot] = spare
    s = dict(case=case, pos=torch.tensor(pos, dtype=torch.int32, device="cuda"), table=table, width=width,
             k_tail=randn(B, Hkv, CHUNK, d), v_tail=randn(B, Hkv, CHUNK, d).to(dt))
    if case["op"] == "append":
        s |= _pages(total + 3, case, gen)
        N = sum(n)
        # The projections' output: q, k and v of a token next to each other.
        qkv = randn(N, Hq + 2 * Hkv, d).to(dt)
        s |= dict(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:],
                  cu=torch.tensor([sum(n[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda"),
                  rope=_table(max(p + m for p, m in zip(pos, n)), case["rot"]), q_out=torch.zeros(N, Hq, d, dtype=dt, device="cuda"))
        return s
    cent = randn(total + 3, Hkv, d)
    s |= _pages(total + 3, case, gen, cent)
    # Each query is near a key of its own context, as trained heads' queries are.
    at = (torch.rand(B, Hkv, device="cuda", generator=gen) * torch.tensor(pages, device="cuda")[:, None]).long()
    page = table.long().gather(1, at.clamp(max=width - 1)).clamp(min=0)
    near = cent[page, torch.arange(Hkv, device="cuda")]
    q = 0.35 * near[:, :, None, :] + 0.5 * randn(B, Hkv, Hq // Hkv, d)
    k_c, k_g = case["k_c"], case["k_g"]
    routed = k_c >= 0
    s |= dict(q=q.view(B, Hq, d).to(dt), O=torch.zeros(B, Hq, d, device="cuda"), lse=torch.zeros(B, Hq, device="cuda"),
              cidx=torch.zeros(B, Hkv, k_c, dtype=torch.int32, device="cuda") if routed else None,
              gidx=torch.zeros(B, Hkv, k_g, dtype=torch.int32, device="cuda") if routed else None)
    return s


# ---- plain forms -----------------------------------------------------------------------

def _rotate(x, c, s, rot, interleaved):
    """x [..., d] float32 with its first rot elements turned by the angles of c, s [..., rot / 2]."""
    if rot == 0:
        return x
    h = rot // 2
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :h], x[..., h:rot])
    ya, yb = a * c - b * s, b * c + a * s
    y = torch.stack([ya, yb], -1).flatten(-2) if interleaved else torch.cat([ya, yb], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _rope_plain(st):
    case, x = st["case"], st["x"].float()
    h = case["rot"] // 2
    t = st["table"][case["pos0"]:case["pos0"] + case["T"]]
    c, s = t[:, :h], t[:, h:]
    if case["back"]:
        return _rotate(x, c, -s, case["rot"], case["interleaved"]).transpose(1, 2).to(TORCH[case["dst"]]).contiguous()
    return _rotate(x.transpose(1, 2), c, s, case["rot"], case["interleaved"]).to(TORCH[case["dst"]]).contiguous()


def _bytes(t):
    """8-bit values as bytes, which every indexing operation takes."""
    return t.view(torch.uint8)


def _append_plain(st):
    case, pos, cu = st["case"], st["pos"].long(), st["cu"].long()
    Hkv, d, rot, h = case["Hkv"], case["d"], case["rot"], case["rot"] // 2
    N, M, B = st["q"].shape[0], sum(_chunks(case)[1]), case["B"]
    n_closed = _chunks(case)[2]
    dev = pos.device
    n = cu[1:] - cu[:-1]
    sid = torch.repeat_interleave(torch.arange(B, device=dev), n, output_size=N)
    t = pos[sid] + torch.arange(N, device=dev) - cu[sid]
    c, s = st["rope"][t][:, None, :h], st["rope"][t][:, None, h:]
    q_out = _rotate(st["q"].float(), c, s, rot, case["interleaved"]).to(st["q"].dtype)
    k = _rotate(st["k"].float(), c, s, rot, case["interleaved"])
    # The touched chunks of each sequence, one after the other, around what the open chunk holds.
    first = pos // CHUNK
    count = (pos + n - 1) // CHUNK - first + 1
    base = count.cumsum(0) - count
    owner = torch.repeat_interleave(torch.arange(B, device=dev), count, output_size=M)
    chunk = first[owner] + torch.arange(M, device=dev) - base[owner]
    wk = torch.zeros(M, CHUNK, Hkv, d, device=dev)
    wv = torch.zeros(M, CHUNK, Hkv, d, device=dev, dtype=st["v"].dtype)
    last = base + count - 1
    wk[base] = wk[last] = st["k_tail"].transpose(1, 2)
    wv[base] = wv[last] = st["v_tail"].transpose(1, 2)
    row = (base[sid] + t // CHUNK - first[sid]) * CHUNK + t % CHUNK
    wk.view(M * CHUNK, Hkv, d)[row] = k
    wv.view(M * CHUNK, Hkv, d)[row] = st["v"]
    st["k_tail"].copy_(wk[last].transpose(1, 2))
    st["v_tail"].copy_(wv[last].transpose(1, 2))
    full = torch.argsort(((chunk + 1) * CHUNK > (pos + n)[owner]).int(), stable=True)[:n_closed]
    page = st["table"].long()[owner[full], chunk[full]]
    gk = wk[full].transpose(1, 2).reshape(n_closed, Hkv, 8, 8, d)
    gv = wv[full].transpose(1, 2).reshape(n_closed, Hkv, 8, 8, d).float()
    if n_closed:
        code, st["k_scale"][page] = _quantise(gk, case["cache"])
        _bytes(st["k_pages"])[page] = _bytes(code).view(n_closed, Hkv, CHUNK, d)
        code, st["v_scale"][page] = _quantise(gv, case["cache"])
        _bytes(st["v_pages"])[page] = _bytes(code).view(n_closed, Hkv, CHUNK, d)
        st["csum"][page] = gk.mean((2, 3))
        st["gsum"][page] = gk.mean(3)
    return _append_out(st, q_out)


def _append_out(st, q_out):
    # The codes come back as they are held: int8 as whole numbers, e4m3 as its values.
    return {k: st[k] for k in ("k_pages", "v_pages", "k_scale", "v_scale", "csum", "gsum", "k_tail", "v_tail")} | dict(q_out=q_out)


def _pick(scores, k, eligible):
    """Ascending indices of the k highest scores, equal ones to the lower index; -1 where there are fewer."""
    scores = torch.where(eligible, scores, torch.full_like(scores, -math.inf))
    n = scores.shape[-1]
    if n < k:
        scores = torch.cat([scores, torch.full_like(scores[..., :1], -math.inf).expand(*scores.shape[:-1], k - n)], -1)
    order = torch.sort(scores, dim=-1, descending=True, stable=True).indices[..., :k]
    some = torch.minimum(eligible.sum(-1, keepdim=True), torch.tensor(k, device=scores.device))
    at = torch.where(torch.arange(k, device=scores.device) < some, order, torch.full_like(order, 1 << 40))
    at = at.sort(-1).values
    return torch.where(at < (1 << 40), at, torch.full_like(at, -1))


def _decode_plain(st):
    case, pos, q = st["case"], st["pos"].long(), st["q"].float()
    B, Hkv, d, G = case["B"], case["Hkv"], case["d"], case["Hq"] // case["Hkv"]
    dev = pos.device
    c0 = torch.div(pos.clamp(min=0), CHUNK, rounding_mode="floor")
    rows = torch.where(pos >= 0, pos % CHUNK + 1, torch.zeros_like(pos))
    C = max(st["width"] - 1, 1)                               # chunks that any sequence has closed
    table = st["table"].long()[:, :C].clamp(min=0)
    C = table.shape[1]
    head = torch.arange(Hkv, device=dev)
    q = q.view(B, Hkv, G, d)
    if case["k_c"] < 0:
        cidx = gidx = None
        page, grp, h = table[:, None, :, None], torch.arange(8, device=dev), head[:, None, None]
        live = (torch.arange(C, device=dev) < c0[:, None])[:, None, :, None].expand(B, Hkv, C, 8).reshape(B, Hkv, C * 8)
    else:
        qs = q.double().sum(2)
        score = torch.einsum("bhd,bchd->bhc", qs, st["csum"][table].double())
        cidx = _pick(score, case["k_c"], (torch.arange(C, device=dev) < c0[:, None])[:, None].expand(B, Hkv, C))
        at = cidx.clamp(min=0)
        cp = table.gather(1, at.view(B, -1)).view(at.shape)
        score = torch.einsum("bhd,bhced->bhce", qs, st["gsum"][cp, head[:, None]].double())
        ok = (cidx >= 0)[..., None].expand(score.shape)
        pick = _pick(score.flatten(-2), case["k_g"], ok.flatten(-2))
        ids = (at[..., None] * 8 + torch.arange(8, device=dev)).flatten(-2)
        gidx = torch.where(pick >= 0, ids.gather(-1, pick.clamp(min=0)), pick)
        at = gidx.clamp(min=0)
        page, grp, h = table.gather(1, (at // 8).view(B, -1)).view(at.shape), at % 8, head[:, None]
        live = gidx >= 0

    def held(name):
        code = _bytes(st[name + "_pages"]).view(-1, Hkv, 8, 8, d)[page, h, grp].view(TORCH[case["cache"]]).float()
        x = code * st[name + "_scale"][page, h, grp][..., None, None]
        return x.reshape(B, Hkv, -1, d)

    live = torch.cat([live[..., None].expand(*live.shape, 8).flatten(-2),
                      (torch.arange(CHUNK, device=dev) < rows[:, None])[:, None].expand(B, Hkv, CHUNK)], -1)
    k = torch.cat([held("k"), st["k_tail"]], 2)
    s = torch.einsum("bhgd,bhtd->bhgt", q, k) * (1.0 / math.sqrt(d))
    del k
    s = torch.where(live[:, :, None], s, torch.full_like(s, -math.inf))
    v = torch.cat([held("v"), st["v_tail"].float()], 2)
    v = torch.where(live[..., None], v, torch.zeros_like(v))
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = (s - m).exp()
    l = p.sum(-1, keepdim=True)
    O = torch.einsum("bhgt,bhtd->bhgd", p, v) / torch.where(l > 0, l, torch.ones_like(l))
    whole = lambda x: None if x is None else x.int()  # noqa: E731
    return dict(O=O.reshape(B, case["Hq"], d), lse=(m + l.log()).view(B, case["Hq"]), cidx=whole(cidx), gidx=whole(gidx))


# ---- one pass ------------------------------------------------------------------------------

def run(state):
    case = state["case"]
    if not own:
        return dict(append=_append_plain, decode=_decode_plain, rope=_rope_plain)[case["op"]](state)
    import hierarchical_routed_sparse_b200 as hga
    if case["op"] == "rope":
        turn = hga.rope_bwd if case["back"] else hga.rope_fwd
        turn(state["x"], state["y"], state["table"], pos0=case["pos0"], interleaved=case["interleaved"])
        return state["y"]
    cache = state.get("handle")
    if cache is None:                      # the cache object that a program makes once and keeps
        p = hga.PagedParams(B=case["B"], Hq=case["Hq"], Hkv=case["Hkv"], d=case["d"], n_pages=state["k_pages"].shape[0],
                            max_chunks=state["width"], k_c=case.get("k_c", -1), k_g=case.get("k_g", -1),
                            dtype=hga.HGA_BF16 if case["dtype"] == "bf16" else hga.HGA_FP32,
                            cache_dtype=hga.HGA_INT8 if case["cache"] == "int8" else hga.HGA_E4M3)
        names = ("k_pages", "v_pages", "k_scale", "v_scale", "csum", "gsum", "k_tail", "v_tail", "table")
        cache = state["handle"] = hga.PagedCache(p, **{k: state[k] for k in names})
    if case["op"] == "append":
        cache.append(state["pos"], state["k"], state["v"], cu=state["cu"], q=state["q"], q_out=state["q_out"],
                     rope=state["rope"], interleaved=case["interleaved"])
        return _append_out(state, state["q_out"])
    cache.decode(state["pos"], state["q"], state["O"], state["lse"], state["cidx"], state["gidx"])
    return {k: state[k] for k in ("O", "lse", "cidx", "gidx")}


# ---- the definitions in 64 bits ---------------------------------------------------------

def _turned(x, angles, rot, interleaved, sign=1.0):
    """x [n, H, d] in 64 bits, pair by pair, with a rotation matrix for each pair."""
    y = x.clone()
    h = rot // 2
    for i in range(h):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
        c, s = angles[:, i, None], sign * angles[:, h + i, None]
        y[..., a] = c * x[..., a] - s * x[..., b]
        y[..., b] = s * x[..., a] + c * x[..., b]
    return y


def _exact_append(st):
    case = st["case"]
    pos, n = _layout(case)
    Hkv, d, rot, inter, top = case["Hkv"], case["d"], case["rot"], case["interleaved"], LEVEL[case["cache"]]
    out = {k: st[k].double() for k in ("k_scale", "v_scale", "csum", "gsum", "k_tail", "v_tail")}
    for name in ("k_pages", "v_pages"):
        out[name] = None if case["cache"] == "int8" else st[name].double()
    q_out, at = [], 0
    for b in range(case["B"]):
        new = slice(at, at + n[b])
        at += n[b]
        ang = st["rope"][pos[b]:pos[b] + n[b]].double()
        q_out.append(_turned(st["q"][new].double(), ang, rot, inter))
        off, first = pos[b] % CHUNK, pos[b] // CHUNK
        k = torch.cat([st["k_tail"][b, :, :off].double().transpose(0, 1), _turned(st["k"][new].double(), ang, rot, inter)])
        v = torch.cat([st["v_tail"][b, :, :off].transpose(0, 1), st["v"][new]]).double()
        full = k.shape[0] // CHUNK
        kept = (k.shape[0] - 1) // CHUNK * CHUNK
        out["k_tail"][b, :, :k.shape[0] - kept] = k[kept:].transpose(0, 1)
        out["v_tail"][b, :, :k.shape[0] - kept] = v[kept:].transpose(0, 1)
        if not full:
            continue
        page = st["table"][b, first:first + full].long()
        for name, x in (("k", k), ("v", v)):
            x = x[:full * CHUNK].view(full, 8, 8, Hkv, d).permute(0, 3, 1, 2, 4)
            big = x.abs().flatten(-2).max(-1).values.clamp(min=top * TINY)
            out[name + "_scale"][page] = big / top
            if case["cache"] == "e4m3":
                held = (x / big[..., None, None] * top).to(torch.float8_e4m3fn).double()
                out[name + "_pages"][page] = held.reshape(full, Hkv, CHUNK, d)
            if name == "k":
                out["gsum"][page] = x.sum(3) / 8
                out["csum"][page] = x.sum((2, 3)) / 64
    return out | dict(q_out=torch.cat(q_out))


def _exact_decode(st):
    case = st["case"]
    pos, _ = _layout(case)
    Hkv, G, d, k_c, k_g = case["Hkv"], case["Hq"] // case["Hkv"], case["d"], case["k_c"], case["k_g"]
    O = torch.zeros(case["B"], Hkv, G, d, dtype=torch.float64, device="cuda")
    lse = torch.full((case["B"], Hkv, G), -math.inf, dtype=torch.float64, device="cuda")
    cidx = gidx = None
    if k_c >= 0:
        cidx = torch.full((case["B"], Hkv, k_c), -1, dtype=torch.int32, device="cuda")
        gidx = torch.full((case["B"], Hkv, k_g), -1, dtype=torch.int32, device="cuda")
    for b, p in enumerate(pos):
        if p < 0:
            continue
        c0, rows = p // CHUNK, p % CHUNK + 1
        pages = st["table"][b, :c0].long()
        kt, vt = st["k_tail"][b, :, :rows].double(), st["v_tail"][b, :, :rows].double()
        q = st["q"][b].double().view(Hkv, G, d)
        for h in range(Hkv):
            groups = torch.arange(8 * c0, device="cuda")
            if k_c >= 0:
                u = q[h].sum(0)
                best = torch.argsort(st["csum"][pages, h].double() @ u, descending=True, stable=True)[:k_c]
                mine = best.sort().values
                cidx[b, h, :len(mine)] = mine.int()
                groups = (mine[:, None] * 8 + torch.arange(8, device="cuda")).flatten()
                best = torch.argsort(st["gsum"][pages[mine], h].double().view(-1, d) @ u, descending=True, stable=True)[:k_g]
                groups = groups[best.sort().values]
                gidx[b, h, :len(groups)] = groups.int()
            kv = []
            for name, tail in (("k", kt), ("v", vt)):
                at, g = pages[groups // 8], groups % 8
                code = st[name + "_pages"][at, h].view(torch.uint8).view(-1, 8, 8, d)[torch.arange(len(groups)), g]
                x = code.view(TORCH[case["cache"]]).double() * st[name + "_scale"][at, h, g].double()[:, None, None]
                kv.append(torch.cat([x.reshape(-1, d), tail[h]]))
            s = q[h] @ kv[0].T / math.sqrt(d)
            lse[b, h] = s.logsumexp(-1)
            O[b, h] = (s - lse[b, h][:, None]).exp() @ kv[1]
    return dict(O=O.view(case["B"], -1, d), lse=lse.view(case["B"], -1), cidx=cidx, gidx=gidx)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(st)
    if case["op"] == "decode":
        return _exact_decode(st)
    x = st["x"].double().transpose(1, 2) if case["back"] else st["x"].double()
    ang = st["table"][case["pos0"]:].double()
    y = torch.stack([_turned(xb, ang, case["rot"], case["interleaved"], -1.0 if case["back"] else 1.0) for xb in x])
    return y if case["back"] else y.transpose(1, 2).contiguous()
