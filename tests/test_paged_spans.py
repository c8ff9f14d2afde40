"""Paged decode where a warp walks a long run of tiles, against float64; and
the order of a captured step.

The split kernel has at most 3 x 148 CTAs of 4 warps, whatever the batch, so
that a large batch gives a warp hundreds of 16-key tiles.

Tolerances.  A row's channel is a sum of terms p D v.  Each term is off by
  - its logit's error: a float32 sum of Dk exact products (on tensor cores, whose
    sums truncate: 2^-23 a step of 8 or 16 channels) times the scale: at most
    Dk/8 2^-23 sum |q k| scale, and 2^-23 of the logit for the two roundings of
    the scale in log2 units;
  - its decay's: 2^-23 of the gates' sum in log2 units for the two roundings of
    that sum, and a tile's 16 additions, 16 2^-24 of the tile's own sum;
  - the exponentials (2 ulp each) and the products' parts: 8 x 2^-23.
Those are taken as they stand.  The float32 sums over n tiles round to nearest,
so their errors are as often up as down: an addition's is spread evenly over at
most 2^-24 of the sum either way, so that their spread is 2^-24 sqrt(n/3); 4
spreads are allowed.  The denominator's sum is compensated and has 2^-23.
All are relative to the sum of the terms' magnitudes (for y: through the norm or
the denominator, which adds as much again)."""
import math

import pytest
import torch

from gated_softmax_attention_fp32_b200 import fixattn

bf16 = torch.bfloat16


def make(lens, Hq, Hkv, Dk, Dv, page, scalar, gate, value=None, qscale=1.0, seed=0):
    """q, pages, table, lengths and weight, made on the GPU; pages in a random order."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-n // page) for n in lens]
    P = sum(need) + 1
    normal = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=bf16)  # noqa: E731
    k, v = normal(P, page, Hkv, Dk), normal(P, page, Hkv, Dv)
    if value is not None:
        v = value(v)
    shape = (P, page, Hkv) if scalar else (P, page, Hkv, Dv)
    g = gate(torch.randn(shape, generator=gen, device="cuda"))
    order = torch.randperm(P, generator=gen, device="cuda").int()
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    q = (normal(len(lens), Hq, Dk).float() * qscale).to(bf16)
    w = (1 + 0.1 * torch.randn(Dv, generator=gen, device="cuda")).to(bf16)
    return q, k, v, g, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), w


def check(y, q, k, v, g, table, lens, w, norm, span, rows, eps=1e-6):
    """Rows `rows` of y (float32) against float64, `span` tiles of 16 keys being walked by a warp at most."""
    Hq, Dk, Hkv = q.shape[1], q.shape[2], k.shape[2]
    assert bool(torch.isfinite(y).all())
    for b in rows:
        L = int(lens[b])
        if L == 0:
            assert not y[b].any()
            continue
        t = table[b, :-(-L // k.shape[1])].long()
        there = (t >= 0).repeat_interleave(k.shape[1])[:L]            # tokens of missing pages are left out
        kb, vb, gb = (x[t.clamp(min=0)].flatten(0, 1)[:L][there].double() for x in (k, v, g))
        after = torch.zeros_like(gb)
        after[:-1] = gb[1:].flip(0).cumsum(0).flip(0)
        if after.dim() == 2:
            after, gb = after[..., None], gb[..., None]
        for h in range(Hq):
            kv = h * Hkv // Hq
            qh = q[b, h].double()
            s = kb[:, kv] @ qh * Dk ** -0.5
            p = (s - s.max()).exp()
            terms = p[:, None] * after[:, kv].exp() * vb[:, kv]
            logit = (kb[:, kv].abs() @ qh.abs()) * Dk ** -0.5 * (Dk / 8) * 2 ** -23 + (s - s.max()).abs() * 2 ** -22
            logit = logit + s.abs() * 2 ** -22
            decay = after[:, kv].abs() * 2 ** -22 + 16 * 16 * gb[:, kv].abs().max() * 2 ** -23
            each = logit[:, None] + decay + 8 * 2 ** -23
            o, size = terms.sum(0), terms.abs()
            err = (size * each).sum(0) + 4 * math.sqrt(span / 3) * 2 ** -24 * size.sum(0)
            if norm:
                f = 1 / (o.square().mean() + eps).sqrt()
                rel = float((f * f * (o.abs() * err).mean()))         # of the factor itself
                ref, bar = o * f * w.double(), (err * f + o.abs() * f * rel) * w.double().abs()
            else:
                den = p.sum()
                rel = float((p * logit).sum() / den) + 9 * 2 ** -23
                ref, bar = o / den, err / den + o.abs() / den * rel
            bar = bar + ref.abs() * 2 ** -22
            got = y[b, h].double()
            ratio = float((got - ref).norm() / bar.norm())
            assert ratio <= 1, (b, h, L, ratio, float((got - ref).norm() / ref.norm()))


def workers(Hq, Hkv):
    return 148 * (3 if Hq // Hkv <= 8 else 2) * 4


def both_norms(args, span, rows):
    for norm in (True, False):
        y = fixattn.fix_attn_decode_paged(*args, y_dtype=torch.float32, o_norm=norm)
        check(y, *args, norm, span, rows)


@pytest.mark.gpu
@pytest.mark.parametrize("scalar", [False, True])
@pytest.mark.parametrize("value", [None, torch.abs], ids=["signed", "positive"])
def test_sums_over_many_tiles_do_not_drift(cuda_lib, scalar, value):
    """No gates: what is left is the softmax's and the values' sums, over the 512 tiles of whole sequences."""
    B, L = 1800, 8192
    assert B >= workers(1, 1)
    args = make([L] * B, 1, 1, 16, 16, 64, scalar, torch.zeros_like, value)
    both_norms(args, L // 16, (0, 1, B // 2, B - 1))


@pytest.mark.gpu
@pytest.mark.parametrize("scalar", [False, True])
@pytest.mark.parametrize("B,L,gate", [(1800, 32768, 1e-4), (1800, 32768, 4.54e-5), (1800, 32768, 1e-5), (2, 131071, 1e-5)])
def test_steady_gates_over_many_tiles(cuda_lib, scalar, B, L, gate):
    """The same small gate at every token (1e-4, and logsigmoid(10) = -4.54e-5): all roundings of a running sum of
    them go the same way.  One warp walks 2048 tiles, or the pieces of some 888 warps are joined."""
    tiles = L // 16 if B > 2 else -(-2 * 8192 // workers(1, 1))
    args = make([L] * B, 1, 1, 16, 16, 64, scalar, lambda x: torch.full_like(x, -gate), torch.abs, 0.25,
                1)
    both_norms(args, tiles, (0, B // 2, B - 1))


@pytest.mark.gpu
@pytest.mark.parametrize("scalar", [False, True])
@pytest.mark.parametrize("top", [0.5, 8.0])
def test_slowly_rising_logits(cuda_lib, scalar, top):
    """Logits that rise evenly by `top` from the newest key to the oldest: the maximum moves at every tile, and all
    weights of a tile are nearly equal, so that the sum of the weights rounds the same way for long."""
    B, L, page = 1800, 32768, 64
    q, k, *rest = args = make([L] * B, 1, 1, 16, 16, page, scalar, torch.zeros_like, torch.abs, seed=2)
    rows = (0, B // 2, B - 1)
    x = torch.arange(L, device="cuda").flip(0).double() / L * top
    k[:, :, :, :2] = 0
    for b in rows:                                          # as a sum of two bf16 channels, 16 bits
        t = rest[2][b].long()
        k[t] = 0
        k[t, :, 0, 0] = x.to(bf16).view(-1, page)
        k[t, :, 0, 1] = (x - x.to(bf16).double()).to(bf16).view(-1, page)
    q.zero_()
    q[:, :, :2] = 4.0                                       # and a scale of 1/4
    both_norms(args, L // 16, rows)


def line(lens, Hq, Hkv):
    """Positions of the split kernel's line: a unit's tiles and 3 more, units of up to 8 or 16 q heads."""
    grp = Hq // Hkv
    blocks = -(-grp // (8 if grp <= 8 else 16))
    return Hkv * blocks * sum(-(-n // 16) + 3 for n in lens if n)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,Dk,Dv,page", [
    (4, 2, 128, 128, 64), (6, 1, 64, 128, 24), (16, 1, 128, 128, 16), (24, 2, 32, 128, 5),
    (8, 1, 64, 64, 16), (2, 2, 128, 64, 7), (9, 1, 64, 64, 48), (20, 1, 16, 64, 16),
    (3, 1, 32, 32, 16), (5, 1, 64, 32, 100), (12, 1, 32, 32, 9), (10, 1, 128, 32, 32),
    (1, 1, 16, 16, 64), (4, 4, 128, 16, 3), (16, 1, 16, 16, 16), (11, 1, 32, 16, 20)])
@pytest.mark.parametrize("scalar", [False, True])
def test_every_variant_over_many_tiles(cuda_lib, Hq, Hkv, Dk, Dv, page, scalar):
    """Each combination of head dim, gate, one or two column blocks and Dk = Dv or not, with a dozen tiles a warp and
    more: whole and cut units, spans of unequal lengths, pages that end inside a tile and a page that is not there.
    Values of one sign and small logits, so that the bar is a few 1e-6 of y."""
    lens = [1, 15, 16, 17, 160, 0, 333, 500] * 40 + [40000, 39999, 16 * 1300, 4097]
    n = workers(Hq, Hkv)
    lens += [30011] * max(0, -(-(13 * n - line(lens, Hq, Hkv)) // line([30011], Hq, Hkv)))
    total = line(lens, Hq, Hkv)
    assert total // n >= 12 and total % n
    args = make(lens, Hq, Hkv, Dk, Dv, page, scalar,
                lambda x: torch.nn.functional.logsigmoid(x + 9), torch.abs, 0.25, Dk + Dv)
    table = args[4]
    for b in (6, len(lens) - 3):
        table[b, lens[b] // page // 2] = -1
    rows = list(range(8)) + [101, 199] + list(range(320, 324)) + [len(lens) - 3, len(lens) - 1]
    both_norms(args, total // n + 1, rows)


# ------------------------------------------------------------------ order of a captured step
@pytest.mark.gpu
@pytest.mark.parametrize("between", ["copy", "clear", "other stream", "nothing"])
def test_captured_step_waits_for_what_it_reads(cuda_lib, between):
    """Append and decode, captured behind a memory copy, a clear, a join of two streams, or each other.  Before each
    replay everything that the step must write or overwrite first holds other data: the new tokens' slots NaN, the
    inputs those of another step, the lengths zero.  A kernel that ran ahead would show them."""
    B, Hq, Hkv, D, page = 3, 8, 2, 64, 16
    gen = torch.Generator(device="cuda").manual_seed(3)
    normal = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=bf16)  # noqa: E731
    lens = torch.tensor([30, 77, 500], dtype=torch.int32, device="cuda")
    cols = 500 // page + 2
    table = torch.randperm(B * cols, generator=gen, device="cuda").int().view(B, cols)
    pages = [normal(B * cols, page, Hkv, D), normal(B * cols, page, Hkv, D),
             -torch.rand(B * cols, page, Hkv, D, generator=gen, device="cuda")]
    f = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda()
    w = torch.ones(D, dtype=bf16, device="cuda")
    src = dict(q=normal(B, 1, Hq, D), k=normal(B, 1, Hkv, D), v=normal(B, 1, Hkv, D),
               g=-torch.rand(B, 1, Hkv, D, generator=gen, device="cuda"), lens=lens)
    inp = {name: x.clone() for name, x in src.items()}
    side, main = torch.cuda.Stream(), torch.cuda.Stream()

    def bring(names):
        if between == "copy":
            for name in names:
                inp[name].copy_(src[name])
        elif between == "clear":
            inp["k"].zero_()
        elif between == "other stream":
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                for name in names:
                    torch.add(src[name], 0, out=inp[name])
            torch.cuda.current_stream().wait_stream(side)

    def step():
        bring(("k", "v", "g", "lens"))
        q, _ = fixattn.fix_attn_append_paged(inp["k"], inp["v"], inp["g"], *pages, table, inp["lens"], q=inp["q"],
                                             inv_freq=f)
        bring(("lens",))
        return fixattn.fix_attn_decode_paged(q[:, 0], *pages, table, inp["lens"], w, y_dtype=torch.float32)

    def spoil():
        for b in range(B):
            n = int(lens[b]) - 1
            for x in pages:
                x[int(table[b, n // page]), n % page] = float("nan")
        if between in ("copy", "other stream"):
            for name in ("k", "v", "g"):
                inp[name].fill_(float("nan"))
            inp["lens"].zero_()
        elif between == "clear":
            inp["k"].fill_(float("nan"))

    main.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(main):
        step()                                             # (a first run outside the graph)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        y = step()
    seen = []
    for i in range(4):
        for name in ("q", "k", "v"):
            src[name].copy_(normal(*src[name].shape))
            inp[name].copy_(src[name])
        spoil()
        want = step().clone()
        filled = [x.clone() for x in pages]
        torch.cuda.synchronize()
        spoil()
        y.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert bool(torch.isfinite(want).all()) and torch.equal(y, want)
        assert all(torch.equal(a, b) for a, b in zip(pages, filled))
        seen.append(want)
    assert not torch.equal(seen[0], seen[1])
