"""Paged decode where a warp walks a long run of tiles, against float64.

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
most 2^-24 of the sum either way, so that their spread is 2^-24 sqrt(n/3) (and
sqrt(2n/3) for the denominator, two additions a tile); 4 spreads are allowed.
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
    Hq, Dk, Hkv, worst = q.shape[1], q.shape[2], k.shape[2], 0.0
    assert bool(torch.isfinite(y).all())
    for b in rows:
        L = int(lens[b])
        if L == 0:
            assert not y[b].any()
            continue
        t = table[b, :-(-L // k.shape[1])].long()
        kb, vb, gb = (x[t].flatten(0, 1)[:L].double() for x in (k, v, g))
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
                rel = float((p * logit).sum() / den) + 4 * math.sqrt(2 * span / 3) * 2 ** -24 + 8 * 2 ** -23
                ref, bar = o / den, err / den + o.abs() / den * rel
            bar = bar + ref.abs() * 2 ** -22
            got = y[b, h].double()
            ratio = float((got - ref).norm() / bar.norm())
            worst = max(worst, ratio)
            assert ratio <= 1, (b, h, L, ratio, float((got - ref).norm() / ref.norm()))
    return worst


def workers(Hq, Hkv):
    return 148 * (3 if Hq // Hkv <= 8 else 2) * 4


def both_norms(args, span, rows):
    for norm in (True, False):
        y = fixattn.fix_attn_decode_paged(*args, y_dtype=torch.float32, o_norm=norm)
        worst = check(y, *args, norm, span, rows)
        print("norm" if norm else "no norm", "%.2f of the bar" % worst)


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
