"""Calls of the rotation and the paged cache at the edges of what they allow:
many heads (a token in several parts), several threads, frozen leaves, one
tensor in two places.  Tolerances as in test_paged.py: a bf16 rounding is off
by 2^-8 of the value at most, a rotated channel by 1e-6 (|a| + |b|) besides."""
import threading

import pytest
import torch

from gated_softmax_attention_fp32_b200 import fixattn

bf16 = torch.bfloat16


def freqs(rot):
    return (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()


def turned(x, pos, f, back=False):
    """x [N,H,D] at positions pos [N], pairs (i, i + D/2): float64, and |a| + |b|."""
    t = pos.double().cuda()[:, None, None] * f.double() * (-1 if back else 1)
    a, b = x.double().chunk(2, -1)
    size = a.abs() + b.abs()
    return torch.cat((a * t.cos() - b * t.sin(), a * t.sin() + b * t.cos()), -1), torch.cat((size, size), -1)


def close(got, ref, size):
    err = (got.double() - ref).abs()
    assert bool((err <= 2.0 ** -8 * ref.abs() + 1e-6 * size).all()), float(err.max())


def normal(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda", dtype=bf16)


@pytest.mark.gpu
@pytest.mark.parametrize("N,Hq,Hkv", [(3, 96, 48), (1, 300, 100), (700, 64, 64)])
def test_rotation_of_many_heads(cuda_lib, N, Hq, Hkv):
    D = 128
    q, k, f = normal(1, 1, N, Hq, D), normal(2, 1, N, Hkv, D), freqs(D)
    pos = torch.arange(N) * 1001
    at = pos.int()[None].cuda()
    qr, kr = fixattn.fix_attn_rotary(q, k, f, positions=at)
    for x, r in ((q, qr), (k, kr)):
        close(r[0], *turned(x[0], pos, f))
    qi, ki = q.clone(), k.clone()
    fixattn.fix_attn_rotary(qi, ki, f, positions=at, out=(qi, ki))
    assert torch.equal(qi, qr) and torch.equal(ki, kr)


@pytest.mark.gpu
@pytest.mark.parametrize("scalar", [False, True])
@pytest.mark.parametrize("Hkv", [33, 100])
def test_append_and_decode_of_many_kv_heads(cuda_lib, scalar, Hkv):
    B, D, page, lens = 3, 64, 16, [40, 1, 0]
    f = freqs(D)
    shape = (8, page, Hkv)
    kp, vp = normal(1, *shape, D), normal(2, *shape, D)
    gp = -torch.rand(*shape, *(() if scalar else (D,)), device="cuda")
    before = [x.clone() for x in (kp, vp, gp)]
    table = torch.tensor([[6, 1, 3], [0, -1, -1], [-1, -1, -1]], dtype=torch.int32, device="cuda")
    seqlens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q, k, v = normal(3, B, 1, 2 * Hkv, D), normal(4, B, 1, Hkv, D), normal(5, B, 1, Hkv, D)
    g = -torch.rand(B, 1, Hkv, *(() if scalar else (D,)), device="cuda")
    qr, kr = fixattn.fix_attn_append_paged(k, v, g, kp, vp, gp, table, seqlens, q=q, inv_freq=f, return_k=True)
    pos = torch.tensor([39, 0, 0])
    close(qr[:, 0], *turned(q[:, 0], pos, f))
    close(kr[:, 0], *turned(k[:, 0], pos, f))
    for old, new, x in zip(before, (kp, vp, gp), (kr, v, g)):
        old[3, 7], old[0, 0] = x[0, 0], x[1, 0]
        assert torch.equal(old, new)
    w = torch.ones(D, dtype=bf16, device="cuda")
    y = fixattn.fix_attn_decode_paged(qr[:, 0], kp, vp, gp, table, seqlens, w, y_dtype=torch.float32)
    assert not y[2].any()
    for b, L in ((0, 40), (1, 1)):
        t = table[b, :-(-L // page)].long()
        kb, vb, gb = (x[t].flatten(0, 1)[:L].double() for x in (kp, vp, gp))
        after = torch.zeros_like(gb)
        after[:-1] = gb[1:].flip(0).cumsum(0).flip(0)
        after = after[..., None] if scalar else after
        s = torch.einsum("hgd,lhd->hgl", qr[b, 0].double().view(Hkv, 2, D), kb) * D ** -0.5
        o = torch.einsum("hgl,lhd->hgd", (s - s.amax(-1, keepdim=True)).exp(), after.exp() * vb)
        ref = (o / (o.square().mean(-1, keepdim=True) + 1e-6).sqrt()).view(2 * Hkv, D)
        assert float(((y[b].double() - ref).norm(dim=1) / ref.norm(dim=1)).max()) <= 1e-4


@pytest.mark.gpu
def test_threads_on_streams_of_their_own(cuda_lib):
    """Calls from several threads at once, each with its stream, cache and gradient."""
    D, page, f, w = 64, 16, freqs(64), torch.ones(64, dtype=bf16, device="cuda")

    def work(seed, out):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            B, P = 3, 40
            kp, vp = normal(seed, P, page, 2, D), normal(seed + 1, P, page, 2, D)
            gp = -torch.rand(P, page, 2, D, device="cuda", generator=torch.Generator("cuda").manual_seed(seed))
            table = torch.arange(36, dtype=torch.int32, device="cuda").view(B, 12)
            seqlens = torch.tensor([5, 100, 180], dtype=torch.int32, device="cuda")
            for _ in range(10):
                q = normal(seed + 2, B, 1, 8, D).requires_grad_(True)
                k = normal(seed + 3, B, 1, 2, D).requires_grad_(True)
                qr, kr = fixattn.fix_rotary(q, k, f, positions=seqlens[:, None])
                dq, dk = torch.autograd.grad((qr, kr), (q, k), (torch.ones_like(qr), torch.ones_like(kr)))
                seqlens += 1
                qa, _ = fixattn.fix_attn_append_paged(k.detach(), k.detach(), gp[0, :B, :, :][:, None].contiguous(),
                                                      kp, vp, gp, table, seqlens, q=q.detach(), inv_freq=f)
                assert torch.equal(qa, qr.detach())
                out.append((fixattn.fix_attn_decode_paged(qa[:, 0], kp, vp, gp, table, seqlens, w), dq, dk))
        stream.synchronize()

    alone, together = [[] for _ in range(4)], [[] for _ in range(4)]
    for i in range(4):
        work(10 * i, alone[i])
    errors = []

    def guarded(i):
        try:
            work(10 * i, together[i])
        except BaseException as e:  # noqa: BLE001  (a thread's error is raised by the test below)
            errors.append(e)

    threads = [threading.Thread(target=guarded, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for a, b in zip(alone, together):
        assert len(a) == len(b) == 10
        assert all(torch.equal(x, y) for p, r in zip(a, b) for x, y in zip(p, r))


@pytest.mark.gpu
def test_gradient_with_a_frozen_or_a_shared_tensor(cuda_lib):
    N, H, D = 50, 4, 64
    f, pos = freqs(D), torch.arange(N)
    x, y, d1, d2 = (normal(i, 1, N, H, D) for i in range(4))
    for frozen in (0, 1):
        leaves = [t.clone().requires_grad_(i != frozen) for i, t in enumerate((x, y))]
        out = fixattn.fix_rotary(*leaves, f)
        g, = torch.autograd.grad(out, leaves[1 - frozen], (d1, d2))
        close(g[0], *turned((d1, d2)[1 - frozen][0], pos, f, True))
    leaf = x.clone().requires_grad_(True)
    out = fixattn.fix_rotary(leaf, leaf, f)
    assert torch.equal(out[0], out[1])
    g, = torch.autograd.grad(out, leaf, (d1, d2))
    (r1, s1), (r2, s2) = (turned(d[0], pos, f, True) for d in (d1, d2))
    err = (g[0].double() - r1 - r2).abs()             # a rounding of each gradient, and one of their sum
    assert bool((err <= 2.0 ** -8 * (r1.abs() + r2.abs() + (r1 + r2).abs()) * (1 + 2.0 ** -7)
                 + 1e-6 * (s1 + s2)).all())
    with torch.no_grad():
        out = fixattn.fix_rotary(leaf, y, f)
    assert not out[0].requires_grad
