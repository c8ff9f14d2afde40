"""Position rotation, append to a paged cache and decode from it, against
plain float64 implementations.

Tolerances.  A value rounded to bf16 is off by at most 2^-8 of itself
(``BF16``).  A rotated channel a cos t - b sin t carries besides the rounding
of t in [-pi, pi] to float (1.2e-7), the float sine's and cosine's own and those
of the products: 1e-6 (|a| + |b|) in all.
A decode row in float32: a logit is a float32 sum of Dk products, off by at
most Dk 2^-24 sum |q_i k_i| scale (6e-5 at Dk = 128 and standard-normal
inputs, where sum |q_i k_i| scale is about 7), which is the relative error of
its exponential; the value sums add a few 2^-20.  So rows are held to
``F32_ROW`` = 1e-4 of their norm, and to BF16 more where y is bf16.
"""
import ctypes
import math

import pytest
import torch

import synth
from gated_softmax_attention_fp32_b200 import fixattn
from oracle import fix_ref

BF16 = 2.0 ** -8
F32_ROW = 1e-4
NAN = float("nan")
bf16 = torch.bfloat16


# ------------------------------------------------------------------ plain forms, float64 on the CPU
def inv_freq(rot, base=10000.0):
    return (base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float()


def rotate_ref(x, pos, f, interleaved=False, inverse=False):
    """x [N,H,D] at positions pos [N] (None where a token has none) -> float64, and |a| + |b|."""
    out, mag = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64)
    half = f.numel()
    for n, p in enumerate(pos):
        if p is None:
            continue
        for i in range(half):
            t = int(p) * float(f[i].double())
            c, s = math.cos(t), math.sin(t) * (-1 if inverse else 1)
            ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            a, b = x[n, :, ia].double(), x[n, :, ib].double()
            out[n, :, ia], out[n, :, ib] = a * c - b * s, a * s + b * c
            mag[n, :, ia] = mag[n, :, ib] = a.abs() + b.abs()
    return out, mag


def check_rotated(got, x, pos, f, interleaved=False, inverse=False, what=""):
    ref, mag = rotate_ref(x.reshape(-1, *x.shape[-2:]).cpu(), pos, f.cpu(), interleaved, inverse)
    err = (got.reshape(ref.shape).double().cpu() - ref).abs()
    assert bool((err <= BF16 * ref.abs() + 1e-6 * mag).all()), (what, float(err.max()))


def decode_ref(q, k, v, g, w, z, scale, eps, norm):
    """One row, all heads: q [Hq,Dk], k [L,Hkv,Dk], v [L,Hkv,Dv], g [L,Hkv,Dv|1] -> [Hq,Dv]."""
    Hq, L, Hkv, Dv = q.shape[0], k.shape[0], v.shape[1], v.shape[2]
    y = torch.zeros(Hq, Dv, dtype=torch.float64)
    if L == 0:
        return y
    for h in range(Hq):
        kv = h * Hkv // Hq
        s = (k[:, kv].double() @ q[h].double()) * scale
        p = (s - s.max()).exp()
        after = torch.zeros(L, g.shape[2], dtype=torch.float64)
        after[:-1] = g[1:, kv].double().flip(0).cumsum(0).flip(0)
        o = (p[:, None] * after.exp() * v[:, kv].double()).sum(0)
        y[h] = o / ((o * o).mean() + eps).sqrt() * w.double() if norm else o / p.sum()
    if z is not None:
        y = y * z.double() * torch.sigmoid(z.double())
    return y


# ------------------------------------------------------------------ caches
class Cache:
    """A paged cache on the GPU whose unused slots hold NaN, pages in a random order."""

    def __init__(self, lens, Hkv, Dk, Dv, page, seed=0, scalar=False, spare=2, cols=0, fill=True,
                 gate=None):
        gen = torch.Generator().manual_seed(seed)
        S = len(lens)
        need = [-(-n // page) for n in lens]
        self.page, self.lens, self.scalar = page, list(lens), scalar
        P = sum(need) + spare
        order = torch.randperm(P, generator=gen).int()
        self.table = torch.full((S, max(max(need) + 1, cols)), -7, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        gd = () if scalar else (Dv,)
        self.k = torch.full((P, page, Hkv, Dk), NAN, dtype=bf16)
        self.v = torch.full((P, page, Hkv, Dv), NAN, dtype=bf16)
        self.g = torch.full((P, page, Hkv) + gd, NAN)
        self.tok = []
        for b, n in enumerate(lens):
            k = torch.randn(n, Hkv, Dk, generator=gen).to(bf16)
            v = torch.randn(n, Hkv, Dv, generator=gen).to(bf16)
            x = torch.randn(n, Hkv, *gd, generator=gen)
            g = gate(x) if gate else torch.nn.functional.logsigmoid(x + 3)
            self.tok.append((k, v, g))
            if fill:
                for i in range(n):
                    pg, sl = int(self.table[b, i // page]), i % page
                    self.k[pg, sl], self.v[pg, sl], self.g[pg, sl] = k[i], v[i], g[i]

    def cuda(self):
        self.seqlens = torch.tensor(self.lens, dtype=torch.int32).cuda()
        return (self.k.cuda(), self.v.cuda(), self.g.cuda(), self.table.cuda(), self.seqlens)


def decode_inputs(B, Hq, Dk, Dv, seed, gate=False):
    gen = torch.Generator().manual_seed(seed + 1000)
    q = torch.randn(B, Hq, Dk, generator=gen).to(bf16)
    w = (1 + 0.1 * torch.randn(Dv, generator=gen)).to(bf16)
    z = torch.randn(B, Hq, Dv, generator=gen).to(bf16) if gate else None
    return q, w, z


def check_decode(y, c, q, w, z, scale=None, eps=1e-6, norm=True, rows=None):
    f32 = y.dtype == torch.float32
    y = y.double().cpu()
    assert bool(torch.isfinite(y).all())
    for b in range(q.shape[0]) if rows is None else rows:
        k, v, g = c.tok[b]
        ref = decode_ref(q[b], k, v, g[..., None] if c.scalar else g, w,
                         None if z is None else z[b], scale or q.shape[2] ** -0.5, eps, norm)
        for h in range(q.shape[1]):
            err, size = float((y[b, h] - ref[h]).norm()), float(ref[h].norm())
            bar = (F32_ROW + (0 if f32 else BF16)) * size
            assert err <= bar, (b, h, len(k), err, size)
    return y


def dev(x):
    return None if x is None else x.cuda()


# ------------------------------------------------------------------ refusals (CPU)
def _problem(**kw):
    p = fixattn.Problem(batch=2, seqlen=1, num_q_heads=4, num_kv_heads=2, head_dim_k=64,
                        head_dim_v=64, eps=1e-6)
    for key, val in kw.items():
        setattr(p, key, val)
    return p


_BUF = (ctypes.c_uint8 * 4096)()
A = (ctypes.addressof(_BUF) + 15) // 16 * 16


def _cache(**kw):
    c = fixattn.PageCache(16, 8, 4, A, A, A, A, A, None)
    for key, val in kw.items():
        setattr(c, key, val)
    return c


def _rot(**kw):
    r = fixattn.Rotation(A, 64, 0)
    for key, val in kw.items():
        setattr(r, key, val)
    return r


NULL, SHAPE, HEAD, GQA, CU, ALIGN, WS = 1, 2, 3, 4, 5, 6, 7


@pytest.mark.parametrize("kw,rkw,args,code", [
    (dict(head_dim_k=48), {}, {}, HEAD),
    (dict(num_q_heads=3), {}, {}, GQA),
    (dict(batch=0), {}, {}, SHAPE),
    (dict(num_seqs=2), {}, {}, CU),
    (dict(num_q_heads=1 << 21), {}, {}, SHAPE),
    (dict(cu_seqlens=A, num_seqs=2), {}, {}, SHAPE),          # packed wants batch 1
    (dict(cu_seqlens=A, batch=1), {}, {}, CU),                # no sequence count
    (dict(cu_seqlens=A + 4, batch=1, num_seqs=2), {}, {}, ALIGN),
    ({}, dict(rot_dim=24), {}, SHAPE),
    ({}, dict(rot_dim=0), {}, SHAPE),
    ({}, dict(rot_dim=128), {}, SHAPE),
    ({}, dict(inv_freq=None), {}, NULL),
    ({}, dict(inv_freq=A + 2), {}, ALIGN),
    ({}, {}, dict(q=None), NULL),
    ({}, {}, dict(q_out=None), NULL),
    ({}, {}, dict(k_out=None), NULL),
    ({}, {}, dict(q=A + 2), ALIGN),
    ({}, {}, dict(k_out=A + 8), ALIGN),
    ({}, {}, dict(positions=A + 2), ALIGN),
    ({}, {}, dict(qs=248), SHAPE),                            # less than a token's heads
    ({}, {}, dict(qs=260), SHAPE),                            # not a multiple of 8
    ({}, {}, dict(ks=-128), SHAPE),
])
def test_rotary_refusals(kw, rkw, args, code):
    a = dict(positions=None, q=A, qs=0, k=A, ks=0, q_out=A, k_out=A) | args
    lib = fixattn.load()
    s = lib.fix_attn_rotary(ctypes.byref(_problem(**kw)), ctypes.byref(_rot(**rkw)), a["positions"],
                            a["q"], a["qs"], a["k"], a["ks"], a["q_out"], a["k_out"], 0, None)
    assert s == code, fixattn.status_string(s)


BAD_CACHES = [
    (dict(page_size=0), SHAPE), (dict(num_pages=0), SHAPE), (dict(max_pages=0), SHAPE),
    (dict(num_pages=1 << 20, page_size=1 << 12), SHAPE),      # rows beyond 32 bits
    (dict(page_table=None), NULL), (dict(seqlens=None), NULL), (dict(k_pages=None), NULL),
    (dict(v_pages=None), NULL), (dict(g_pages=None), NULL),
    (dict(page_table=A + 2), ALIGN), (dict(k_pages=A + 2), ALIGN), (dict(g_pages=A + 8), ALIGN),
    (dict(status=A + 1), ALIGN),
]


@pytest.mark.parametrize("kw,ckw,args,code", [({}, c, {}, code) for c, code in BAD_CACHES] + [
    (dict(head_dim_v=100), {}, {}, HEAD),
    (dict(flags=8), {}, {}, SHAPE),
    ({}, {}, dict(k=None), NULL),
    ({}, {}, dict(v=None), NULL),
    ({}, {}, dict(g=None), NULL),
    ({}, {}, dict(q=None), NULL),                             # q_out without q
    ({}, {}, dict(r=False), NULL),                            # q without a rotation
    ({}, {}, dict(r=False, q=None, q_out=None), NULL),        # k_out without a rotation
    ({}, {}, dict(v=A + 2), ALIGN),
    ({}, {}, dict(g=A + 4), ALIGN),
    ({}, {}, dict(vs=120), SHAPE),
    ({}, {}, dict(gs=130), SHAPE),
])
def test_append_refusals(kw, ckw, args, code):
    a = dict(r=True, q=A, qs=0, k=A, ks=0, v=A, vs=0, g=A, gs=0, q_out=A, k_out=A) | args
    lib = fixattn.load()
    s = lib.fix_attn_append_paged(
        ctypes.byref(_problem(**kw)), ctypes.byref(_cache(**ckw)),
        ctypes.byref(_rot()) if a["r"] else None, a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"],
        a["g"], a["gs"], a["q_out"], a["k_out"], None)
    assert s == code, fixattn.status_string(s)


@pytest.mark.parametrize("kw,ckw,args,code", [({}, c, {}, code) for c, code in BAD_CACHES] + [
    (dict(seqlen=2), {}, {}, SHAPE),
    (dict(y_dtype=4), {}, {}, 8),
    (dict(eps=-1.0), {}, {}, SHAPE),
    (dict(num_seqs=1), {}, {}, CU),
    (dict(head_dim_v=256), {}, {}, HEAD),
    ({}, {}, dict(q=None), NULL),
    ({}, {}, dict(w=None), NULL),
    ({}, {}, dict(y=None), NULL),
    ({}, {}, dict(ws=None), NULL),
    ({}, {}, dict(q=A + 2), ALIGN),
    ({}, {}, dict(z=A + 4), ALIGN),
    ({}, {}, dict(ws=A + 8), ALIGN),
    ({}, {}, dict(n=16), WS),
])
def test_decode_paged_refusals(kw, ckw, args, code):
    a = dict(q=A, w=A, z=None, y=A, ws=A, n=1 << 40) | args
    lib = fixattn.load()
    p, c = _problem(**kw), _cache(**ckw)
    if code in (SHAPE, HEAD, CU, 8) or ckw:
        assert lib.fix_attn_decode_paged_workspace_bytes(ctypes.byref(p), ctypes.byref(c)) == 0
    s = lib.fix_attn_decode_paged(ctypes.byref(p), ctypes.byref(c), a["q"], a["w"], a["z"], a["y"],
                                  a["ws"], a["n"], None)
    assert s == code, fixattn.status_string(s)


def test_python_refuses_cpu_tensors_and_wrong_kinds():
    q = torch.zeros(1, 2, 2, 64, dtype=bf16)
    with pytest.raises(ValueError, match="CUDA"):
        fixattn.fix_attn_rotary(q, q, inv_freq(64))
    with pytest.raises(ValueError, match="CUDA"):
        fixattn.fix_attn_append_paged(q, q, q.float(), q, q, q.float(), None, None)
    with pytest.raises(ValueError, match="CUDA"):
        fixattn.fix_attn_decode_paged(q[0], q, q, q.float(), None, None)
    with pytest.raises(TypeError):
        fixattn.fix_attn_rotary(None, None, inv_freq(64))


def test_token_strides():
    x = torch.zeros(2, 5, 12, 64)
    f = fixattn._token_stride
    assert f("x", x, 12 * 64) == 12 * 64
    assert f("x", x[:, :, 2:6], 4 * 64) == 12 * 64            # a slice of a fused projection
    assert f("x", x[:1, :, :3], 3 * 64) == 12 * 64
    assert f("x", x[:, :1, :3], 3 * 64) == 5 * 12 * 64        # one token each: the batch's stride
    assert f("x", x[:, :, 0, :8], 8) == 12 * 64               # [B,T,H], as a scalar gate is
    for bad in (x.transpose(1, 2), x[:, :4, :3], x[..., :32], x[:, ::2].flip(0)[:, :, ::2],
                x[:, :, :1].expand(2, 5, 4, 64), x[:1].expand(2, 5, 12, 64)[:, :, :4]):
        with pytest.raises(ValueError, match="evenly spaced"):
            f("x", bad, bad.shape[2] * bad.shape[3])


# ------------------------------------------------------------------ rotation (GPU)
@pytest.mark.gpu
@pytest.mark.parametrize("B,T,Hq,Hkv,D,rot,inter", [
    (1, 1, 1, 1, 16, 16, False), (2, 7, 4, 2, 32, 32, True), (1, 33, 3, 1, 64, 32, True),
    (3, 5, 8, 8, 64, 64, False), (2, 9, 5, 1, 128, 128, False), (1, 4, 2, 2, 128, 48, False),
    (2, 3, 16, 4, 128, 16, True)])
@pytest.mark.parametrize("how", ["plain", "positions", "fused"])
def test_rotary(cuda_lib, B, T, Hq, Hkv, D, rot, inter, how):
    gen = torch.Generator().manual_seed(B * 100 + T)
    qkv = torch.randn(B, T, Hq + Hkv, D, generator=gen).to(bf16)
    q, k = qkv[:, :, :Hq], qkv[:, :, Hq:]
    f = inv_freq(rot)
    positions, pos = None, [t for _ in range(B) for t in range(T)]
    if how == "positions":
        positions = torch.randint(-5, 2**31 - 1, (B, T), generator=gen).int()
        pos = positions.flatten().tolist()
    on = qkv.cuda()
    qd, kd = (on[:, :, :Hq], on[:, :, Hq:]) if how == "fused" else (dev(q).contiguous(), dev(k).contiguous())
    for inverse in (False, True):
        qo, ko = fixattn.fix_attn_rotary(qd, kd, f.cuda(), positions=dev(positions), interleaved=inter,
                                         inverse=inverse)
        # at positions near 2^31 the double product is off by 2^-53 x 2^31 = 2.4e-7 rad, on both sides alike
        check_rotated(qo, q, pos, f, inter, inverse, "q")
        check_rotated(ko, k, pos, f, inter, inverse, "k")
        assert qo.is_contiguous() and ko.is_contiguous()
    assert torch.equal(on.cpu(), qkv)                          # the inputs stay
    only, none = fixattn.fix_attn_rotary(qd, None, f.cuda(), positions=dev(positions),
                                         interleaved=inter, inverse=True)
    assert none is None and torch.equal(only, qo)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,behind", [([5], 0), ([0, 3, 0, 0, 9, 1, 0], 4), ([1] * 70, 0), ([2] * 1100, 3)])
def test_rotary_packed(cuda_lib, lens, behind):
    N, D = sum(lens) + behind, 64
    gen = torch.Generator().manual_seed(N)
    q, k = torch.randn(1, N, 2, D, generator=gen).to(bf16), torch.randn(1, N, 1, D, generator=gen).to(bf16)
    cu = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0)
    pos = [t for n in lens for t in range(n)] + [None] * behind
    f = inv_freq(D)
    qo, ko = fixattn.fix_attn_rotary(q.cuda(), k.cuda(), f.cuda(), cu_seqlens=cu.cuda())
    check_rotated(qo, q, pos, f)
    check_rotated(ko, k, pos, f)
    if behind:
        assert torch.equal(qo[:, -behind:].cpu(), q[:, -behind:])


@pytest.mark.gpu
def test_rotary_in_place_empty_and_other_stream(cuda_lib):
    gen = torch.Generator().manual_seed(5)
    q, k = torch.randn(2, 300, 8, 128, generator=gen).to(bf16), torch.randn(2, 300, 2, 128, generator=gen).to(bf16)
    f = inv_freq(128).cuda()
    want = fixattn.fix_attn_rotary(q.cuda(), k.cuda(), f)
    qi, ki = q.cuda(), k.cuda()
    got = fixattn.fix_attn_rotary(qi, ki, f, out=(qi, ki))
    assert got[0] is qi and torch.equal(qi, want[0]) and torch.equal(ki, want[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fixattn.fix_attn_rotary(q.cuda(), k.cuda(), f, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    e = fixattn.fix_attn_rotary(q.cuda()[:, :0], k.cuda()[:, :0], f)
    assert e[0].shape == (2, 0, 8, 128) and e[1].shape == (2, 0, 2, 128)


@pytest.mark.gpu
@pytest.mark.parametrize("inter,packed", [(False, False), (True, True)])
def test_rotary_gradient(cuda_lib, inter, packed):
    """Against the formula (the rotation back), and against differences: the
    loss is linear in q and k, so between any two points it changes by the
    gradient's product with the step, up to the roundings of the bf16 outputs
    and gradients: BF16 of the sum of the products' magnitudes."""
    gen = torch.Generator().manual_seed(8)
    B, T, Hq, Hkv, D = (1, 40, 4, 2, 64) if packed else (2, 20, 4, 2, 64)
    mk = lambda h: torch.randn(B, T, h, D, generator=gen).to(bf16)  # noqa: E731
    q, k, dq, dk, q2, k2 = (mk(h) for h in (Hq, Hkv) * 3)
    lens = [13, 0, 27]
    cu = torch.tensor([0] + lens).cumsum(0).cuda() if packed else None
    pos = [t for n in (lens if packed else [T] * B) for t in range(n)]
    f = inv_freq(32)
    run = lambda a, b: fixattn.fix_rotary(a, b, f.cuda(), cu_seqlens=cu, interleaved=inter)  # noqa: E731
    ql, kl = q.cuda().requires_grad_(True), k.cuda().requires_grad_(True)
    qr, kr = run(ql, kl)
    gq, gk = torch.autograd.grad((qr, kr), (ql, kl), (dq.cuda(), dk.cuda()))
    check_rotated(qr.detach(), q, pos, f, inter)
    check_rotated(gq, dq, pos, f, inter, True, "dq")
    check_rotated(gk, dk, pos, f, inter, True, "dk")
    q2r, k2r = run(q2.cuda(), k2.cuda())
    for a, b, a2, b2, d, g in ((q, qr, q2, q2r, dq, gq), (k, kr, k2, k2r, dk, gk)):
        change = ((b2.double() - b.detach().double()).cpu() * d.double())
        step = g.double().cpu() * (a2.double() - a.double())
        bar = BF16 * float((change.abs().sum() * 2 + step.abs().sum()))
        assert abs(float(change.sum() - step.sum())) <= bar
    # a gradient that comes expanded, and one output that nothing uses
    gq2, gk2 = torch.autograd.grad(run(ql, kl)[0].sum(), (ql, kl))
    check_rotated(gq2, torch.ones_like(q), pos, f, inter, True, "ones")
    assert not gk2.any()


# ------------------------------------------------------------------ append (GPU)
def expect_append(c, k, v, g, f, inter, pos_seq, before):
    """The pages after the append, float64 keys, and |a| + |b| of each stored key channel."""
    pos = [p for p, _ in pos_seq]
    ref, mag = (rotate_ref(k, [max(p, 0) if p is not None else None for p in pos], f, inter)
                if f is not None else (k.double(), torch.zeros(k.shape, dtype=torch.float64)))
    kp, vp, gp = before[0].double(), before[1].clone(), before[2].clone()
    km = torch.zeros(kp.shape, dtype=torch.float64)
    for n, (p, b) in enumerate(pos_seq):
        if p is None or p < 0 or p // c.page >= c.table.shape[1]:
            continue
        pg, sl = int(c.table[b, p // c.page]), p % c.page
        if 0 <= pg < kp.shape[0]:
            kp[pg, sl], vp[pg, sl], gp[pg, sl], km[pg, sl] = ref[n], v[n], g[n], mag[n]
    return kp, vp, gp, km


@pytest.mark.gpu
@pytest.mark.parametrize("S,T,lens,Hq,Hkv,Dk,Dv,page,scalar,rot,inter", [
    (1, 1, [1], 1, 1, 16, 16, 1, False, 16, False),
    (3, 1, [70, 1, 33], 4, 2, 64, 64, 16, False, 64, False),
    (4, 1, [5, 0, 40, 0], 8, 2, 128, 128, 64, False, 128, False),     # two padding rows
    (2, 5, [5, 18], 4, 1, 32, 128, 3, True, 32, True),
    (3, 4, [2, 9, 100], 6, 3, 128, 32, 24, True, 48, False),          # a short sequence: its first tokens are padding
    (2, 6, [6, 31], 2, 2, 64, 16, 7, False, 0, False),
])
def test_append(cuda_lib, S, T, lens, Hq, Hkv, Dk, Dv, page, scalar, rot, inter):
    gen = torch.Generator().manual_seed(S * 10 + T)
    c = Cache(lens, Hkv, Dk, Dv, page, seed=3, scalar=scalar)
    kp, vp, gp, table, seqlens = c.cuda()
    q = torch.randn(S, T, Hq, Dk, generator=gen).to(bf16)
    k = torch.randn(S, T, Hkv, Dk, generator=gen).to(bf16)
    v = torch.randn(S, T, Hkv, Dv, generator=gen).to(bf16)
    g = -torch.rand(S, T, Hkv, *(() if scalar else (Dv,)), generator=gen)
    f = inv_freq(rot) if rot else None
    # k and v as slices of wider tensors
    wide_k = torch.randn(S, T, Hkv + 2, Dk, generator=gen).to(bf16)
    wide_k[:, :, 1:1 + Hkv] = k
    wide_g = torch.zeros(S, T, Hkv + 1, *g.shape[3:])
    wide_g[:, :, 1:] = g
    pos_seq = [(lens[b] - T + t, b) for b in range(S) for t in range(T)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = expect_append(c, k.flatten(0, 1), v.flatten(0, 1), g.flatten(0, 1), f, inter, pos_seq, (c.k, c.v, c.g))
    gd = wide_g.cuda()[:, :, 1:]
    if not scalar and gd.storage_offset() % 4:
        gd = gd.contiguous()
    qo, ko = fixattn.fix_attn_append_paged(wide_k.cuda()[:, :, 1:1 + Hkv], v.cuda(), gd, kp, vp, gp, table,
                                           seqlens, q=dev(q) if rot else None, inv_freq=dev(f),
                                           interleaved=inter, return_k=rot > 0, status=status)
    assert int(status) == 0
    err = (kp.double().cpu() - want[0]).abs()
    keep = torch.isnan(want[0])
    assert torch.equal(keep, torch.isnan(kp.cpu()))            # nothing else was written
    assert bool((err[~keep] <= (BF16 * want[0].abs() + 1e-6 * want[3])[~keep]).all())
    assert torch.equal(vp.cpu().view(torch.int16), want[1].view(torch.int16))
    assert torch.equal(gp.cpu().view(torch.int32), want[2].view(torch.int32))
    if rot:
        pos = [p if p >= 0 else None for p, _ in pos_seq]
        check_rotated(qo, q, pos, f, inter, what="q")
        check_rotated(ko, k, pos, f, inter, what="k")
    else:
        assert qo is None and ko is None


@pytest.mark.gpu
def test_append_packed_with_rows_behind(cuda_lib):
    """Ragged new tokens, an empty sequence among them, onto caches of other
    lengths; the buffer has room behind the last sequence."""
    new, lens, behind = [3, 0, 17, 1], [10, 4, 17, 64], 5
    Hq, Hkv, D, page = 4, 2, 64, 16
    c = Cache(lens, Hkv, D, D, page, seed=4)
    kp, vp, gp, table, seqlens = c.cuda()
    N = sum(new) + behind
    gen = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(1, N, h, D, generator=gen).to(bf16) for h in (Hq, Hkv, Hkv))
    g = -torch.rand(1, N, Hkv, D, generator=gen)
    cu = torch.tensor([0] + new).cumsum(0)
    pos_seq = [(L - n + t, b) for b, (n, L) in enumerate(zip(new, lens)) for t in range(n)] + [(None, 0)] * behind
    f = inv_freq(D)
    want = expect_append(c, k[0], v[0], g[0], f, False, pos_seq, (c.k, c.v, c.g))
    qo, ko = fixattn.fix_attn_append_paged(k.cuda(), v.cuda(), g.cuda(), kp, vp, gp, table, seqlens,
                                           cu_seqlens=cu.cuda(), q=q.cuda(), inv_freq=f.cuda(), return_k=True)
    keep = torch.isnan(want[0])
    assert torch.equal(keep, torch.isnan(kp.cpu()))
    err = (kp.double().cpu() - want[0]).abs()
    assert bool((err[~keep] <= (BF16 * want[0].abs() + 1e-6 * want[3])[~keep]).all())
    assert torch.equal(vp.cpu().view(torch.int16), want[1].view(torch.int16))
    assert torch.equal(gp.cpu().view(torch.int32), want[2].view(torch.int32))
    check_rotated(qo, q, [p for p, _ in pos_seq], f)
    check_rotated(ko, k, [p for p, _ in pos_seq], f)


@pytest.mark.gpu
def test_missing_pages_are_skipped_and_reported(cuda_lib):
    """Page ids outside the pool and lengths beyond the table: the kernels
    check them before any access, skip the token and set the status."""
    Hkv, D, page = 2, 64, 16
    c = Cache([40, 20], Hkv, D, D, page, seed=6, fill=True)
    good = c.table.clone()
    x = torch.randn(2, 1, Hkv, D, generator=torch.Generator().manual_seed(1)).to(bf16).cuda()
    g = torch.full((2, 1, Hkv, D), -0.5, device="cuda")
    q, w, _ = decode_inputs(2, 4, D, D, 3)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def fresh(table, lens):
        kp, vp, gp, _, _ = c.cuda()
        return kp, vp, gp, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()

    # the last token of sequence 0 lies in a page that is not there
    for bad in (-1, c.k.shape[0], 2**31 - 1, -2**31):
        table = good.clone()
        table[0, 2] = bad
        pages = fresh(table, [40, 20])
        status.zero_()
        fixattn.fix_attn_append_paged(x, x, g, *pages, status=status)
        assert int(status) == fixattn.FIX_ERR_PAGE
        assert torch.equal(pages[0][int(good[1, 1]), 3], x[1, 0])     # sequence 1's token is stored
        diff = (pages[0].cpu().view(torch.int16) != c.k.view(torch.int16)).flatten(2).any(-1)
        assert int(diff.sum()) == 1                                   # and nothing else
        # the decode leaves the page's keys out: as if the sequence ended before it
        pages = fresh(table, [40, 20])
        status.zero_()
        y = fixattn.fix_attn_decode_paged(q.cuda(), *pages, w.cuda(), y_dtype=torch.float32, status=status)
        assert int(status) == fixattn.FIX_ERR_PAGE
        short = fresh(good, [32, 20])
        y2 = fixattn.fix_attn_decode_paged(q.cuda(), *short, w.cuda(), y_dtype=torch.float32)
        assert float((y - y2).norm() / y2.norm()) <= F32_ROW
    # a length beyond the table's columns: the tokens that the table holds count
    pages = fresh(good[:, :2].contiguous(), [40, 20])
    status.zero_()
    y3 = fixattn.fix_attn_decode_paged(q.cuda(), *pages, w.cuda(), y_dtype=torch.float32, status=status)
    assert int(status) == fixattn.FIX_ERR_PAGE
    assert float((y3 - y2).norm() / y2.norm()) <= F32_ROW
    status.zero_()
    fixattn.fix_attn_append_paged(x, x, g, *pages, status=status)
    assert int(status) == fixattn.FIX_ERR_PAGE
    pages = fresh(good, [2**31 - 1, 20])
    status.zero_()
    fixattn.fix_attn_append_paged(x, x, g, *pages, status=status)
    assert int(status) == fixattn.FIX_ERR_PAGE
    # no status word: the same, silently; and a good call leaves the word alone
    fixattn.fix_attn_append_paged(x, x, g, *fresh(good[:, :2].contiguous(), [40, 20]))
    status.fill_(77)
    fixattn.fix_attn_decode_paged(q.cuda(), *fresh(good, [40, 0]), w.cuda(), status=status)
    assert int(status) == 77


# ------------------------------------------------------------------ decode (GPU)
EDGE = [0, 1, 2, 15, 16, 17, 31, 33, 64, 100, 129, 257]


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,Dk,Dv,page,scalar", [
    (1, 1, 16, 16, 1, False), (2, 1, 32, 64, 16, False), (4, 2, 64, 64, 24, False), (6, 2, 128, 128, 64, False),
    (8, 1, 128, 128, 16, False), (9, 1, 64, 128, 5, False), (16, 1, 128, 128, 32, False), (5, 5, 128, 16, 16, False),
    (17, 1, 128, 64, 16, False), (40, 1, 32, 32, 100, False), (3, 1, 16, 128, 64, False),
    (1, 1, 16, 16, 3, True), (4, 2, 64, 64, 16, True), (10, 1, 128, 128, 24, True), (16, 2, 64, 128, 7, True),
    (33, 1, 128, 32, 16, True), (2, 2, 32, 16, 64, True)])
@pytest.mark.parametrize("opts", [dict(), dict(norm=False, gate=True), dict(gate=True, f32=False)])
def test_decode_paged(cuda_lib, Hq, Hkv, Dk, Dv, page, scalar, opts):
    c = Cache(EDGE, Hkv, Dk, Dv, page, seed=Hq + Dk, scalar=scalar)
    norm = opts.get("norm", True)
    q, w, z = decode_inputs(len(EDGE), Hq, Dk, Dv, page, opts.get("gate", False))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = fixattn.fix_attn_decode_paged(q.cuda(), *c.cuda(), w.cuda() if norm else None,
                                      y_dtype=torch.float32 if opts.get("f32", True) else bf16, o_gate=dev(z),
                                      o_norm=norm, status=status)
    assert int(status) == 0
    check_decode(y, c, q, w, z, norm=norm)
    assert not y[0].any()                                       # length 0


@pytest.mark.gpu
@pytest.mark.parametrize("name,gate,qscale,scale", [
    ("no forgetting", lambda x: torch.zeros_like(x), 1, None),
    ("strong", lambda x: -200 * x.abs(), 1, None),
    ("closed gates", lambda x: torch.where(x > 1.5, -math.inf, -0.1 * x.abs()), 1, None),
    ("lowest", lambda x: torch.where(x > 1.5, torch.finfo(torch.float32).min, -0.1 * x.abs()), 1, None),
    ("opening", lambda x: 0.05 * x, 1, None),
    ("sharp logits", lambda x: -0.01 * x.abs(), 16, None),
    ("given scale", lambda x: -0.01 * x.abs(), 1, 0.3)])
@pytest.mark.parametrize("scalar", [False, True])
def test_decode_paged_gates_and_logits(cuda_lib, name, gate, qscale, scale, scalar):
    """Gates that close a channel for good, sums beyond float's exponent
    range, and logits of some hundreds (whose float32 error, 16 times the
    ordinary one, sets the bar there)."""
    lens = [300, 47, 1]
    c = Cache(lens, 2, 64, 128, 16, seed=9, scalar=scalar, gate=gate)
    q, w, _ = decode_inputs(3, 8, 64, 128, 5)
    q = q * qscale
    for norm in (True, False):
        y = fixattn.fix_attn_decode_paged(q.cuda(), *c.cuda(), w.cuda(), scale=scale, y_dtype=torch.float32,
                                          o_norm=norm).double().cpu()
        assert bool(torch.isfinite(y).all())
        for b in range(3):
            k, v, g = c.tok[b]
            ref = decode_ref(q[b], k, v, g[..., None] if scalar else g, w, None, scale or 0.125, 1e-6, norm)
            err = (y[b] - ref).norm(dim=1) / ref.norm(dim=1)
            assert float(err.max()) <= F32_ROW * qscale, (name, b, float(err.max()))


@pytest.mark.gpu
def test_decode_paged_infinities_in_the_cache(cuda_lib):
    """A key of -inf logit (a channel of -inf against a positive query) drops
    out; in a sequence of such keys alone no logit is finite and y is 0; a NaN
    key makes its own sequence NaN and no other."""
    c = Cache([40, 5, 50, 33], 1, 32, 32, 16, seed=2)
    q, w, _ = decode_inputs(4, 4, 32, 32, 7)
    q[:, :, 0] = 1.0
    drop = [3, 17, 39]
    for b, which in ((0, drop), (1, range(5))):
        for i in which:
            c.k[int(c.table[b, i // 16]), i % 16, 0, 0] = -math.inf
    c.k[int(c.table[2, 1]), 4, 0, 5] = NAN
    y = fixattn.fix_attn_decode_paged(q.cuda(), *c.cuda(), w.cuda(), y_dtype=torch.float32).double().cpu()
    k, v, g = (x.clone() for x in c.tok[0])
    k[drop, 0, 0] = -1e30                                       # exp underflows to 0 all the same
    ref = decode_ref(q[0], k, v, g, w, None, 32 ** -0.5, 1e-6, True)
    assert float((y[0] - ref).norm() / ref.norm()) <= F32_ROW
    assert not y[1].any()
    assert bool(torch.isnan(y[2]).all())
    ref = decode_ref(q[3], *c.tok[3], w, None, 32 ** -0.5, 1e-6, True)
    assert float((y[3] - ref).norm() / ref.norm()) <= F32_ROW


@pytest.mark.gpu
@pytest.mark.parametrize("lens,Hq,Hkv,scalar", [
    ([70001], 4, 1, False), ([20000, 3, 900], 16, 2, False), ([33333], 8, 8, True),
    ([1, 5000, 0, 700, 16, 12345, 64], 24, 2, True)])
def test_decode_paged_long(cuda_lib, lens, Hq, Hkv, scalar):
    """Long and unequal caches, where the work of a sequence is split and
    joined; slow gates, so that far tokens count."""
    D, page = 64, 64
    c = Cache(lens, Hkv, D, D, page, seed=11, scalar=scalar, gate=lambda x: -1e-4 * x.abs())
    q, w, _ = decode_inputs(len(lens), Hq, D, D, 13)
    args = c.cuda()
    y = fixattn.fix_attn_decode_paged(q.cuda(), *args, w.cuda(), y_dtype=torch.float32)
    y2 = fixattn.fix_attn_decode_paged(q.cuda(), *args, w.cuda(), y_dtype=torch.float32)
    assert torch.equal(y, y2)                                    # the same bits each time
    check_decode(y, c, q, w, None)


@pytest.mark.gpu
def test_decode_paged_many_sequences(cuda_lib):
    """More sequences than the split has workers, lengths from 0."""
    gen = torch.Generator().manual_seed(0)
    lens = torch.randint(0, 60, (2100,), generator=gen).tolist()
    c = Cache(lens, 1, 16, 16, 8, seed=12)
    q, w, _ = decode_inputs(len(lens), 2, 16, 16, 14)
    y = fixattn.fix_attn_decode_paged(q.cuda(), *c.cuda(), w.cuda(), y_dtype=torch.float32)
    check_decode(y, c, q, w, None, rows=list(range(0, 2100, 37)) + [2099])
    for b in range(2100):
        if lens[b] == 0:
            assert not y[b].any()


@pytest.mark.gpu
def test_decode_paged_agrees_with_the_contiguous_decode(cuda_lib):
    lens, D, page = [1, 70, 300, 129], 64, 16
    c = Cache(lens, 2, D, D, page, seed=21)
    q, w, z = decode_inputs(4, 8, D, D, 22, True)
    kc, vc, gc = torch.zeros(4, 320, 2, D, dtype=bf16), torch.zeros(4, 320, 2, D, dtype=bf16), torch.zeros(4, 320, 2, D)
    for b, (k, v, g) in enumerate(c.tok):
        kc[b, :lens[b]], vc[b, :lens[b]], gc[b, :lens[b]] = k, v, g
    args = c.cuda()
    y = fixattn.fix_attn_decode_paged(q.cuda(), *args, w.cuda(), y_dtype=torch.float32, o_gate=z.cuda())
    ref = fixattn.fix_attn_decode(q.cuda(), kc.cuda(), vc.cuda(), gc.cuda(), args[4], w.cuda(),
                                  y_dtype=torch.float32, o_gate=z.cuda())
    assert float((y - ref).norm() / ref.norm()) <= 2 * F32_ROW


@pytest.mark.gpu
def test_offsets_beyond_32_bits(cuda_lib):
    """A pool of more than 2^31 key channels (and 2^32 bytes of them), with
    the sequence's pages at its far end."""
    Hkv, D, page = 1, 128, 64
    P = 2**31 // (D * page) + 40
    c = Cache([100], Hkv, D, D, page, seed=31)
    kp = torch.empty(P, page, Hkv, D, dtype=bf16, device="cuda")
    vp, gp = torch.empty_like(kp), torch.empty(P, page, Hkv, D, device="cuda")
    table = torch.tensor([[P - 1, P - 30]], dtype=torch.int32)
    for i in range(2):
        for x, y in ((kp, c.k), (vp, c.v), (gp, c.g)):
            x[int(table[0, i])] = y[int(c.table[0, i])].cuda()
    q, w, _ = decode_inputs(1, 4, D, D, 32)
    seqlens = torch.tensor([100], dtype=torch.int32).cuda()
    y = fixattn.fix_attn_decode_paged(q.cuda(), kp, vp, gp, table.cuda(), seqlens, w.cuda(), y_dtype=torch.float32)
    check_decode(y, c, q, w, None)
    x = torch.randn(1, 1, 1, D, generator=torch.Generator().manual_seed(3)).to(bf16).cuda()
    g = torch.full((1, 1, 1, D), -0.25, device="cuda")
    fixattn.fix_attn_append_paged(x, x, g, kp, vp, gp, table.cuda(), seqlens)
    assert torch.equal(kp[P - 30, 35, 0], x.flatten()) and torch.equal(gp[P - 30, 35, 0], g.flatten())


# ------------------------------------------------------------------ calls as a program makes them (GPU)
@pytest.mark.gpu
def test_prompt_then_steps_match_the_oracle(cuda_lib):
    """Prompts: rotate, fix_attn and append in one go; then steps of append
    and decode.  Every row must be the oracle's row of the whole sequence."""
    B, Hq, Hkv, D, page, steps = 2, 4, 2, 64, 16, 5
    prompts = [150, 37]
    case = synth.make_case(B, max(prompts) + steps, Hq, Hkv, D, D, seed=77)
    f = inv_freq(D).cuda()
    on = {x: case[x].cuda() for x in ("q", "k", "v", "g", "w")}
    cols = -(-(max(prompts) + steps) // page)
    table = torch.randperm(B * cols, generator=torch.Generator().manual_seed(1)).int().view(B, cols).cuda()
    kp = torch.full((B * cols, page, Hkv, D), NAN, dtype=bf16, device="cuda")
    vp, gp = kp.clone(), kp.float()
    pack = lambda x: torch.cat([x[b, :n] for b, n in enumerate(prompts)])[None].contiguous()  # noqa: E731
    cu = torch.tensor([0] + prompts).cumsum(0)
    seqlens = torch.tensor(prompts, dtype=torch.int32).cuda()
    pq, pk, pv, pg = (pack(on[x]) for x in ("q", "k", "v", "g"))
    qr, kr = fixattn.fix_attn_append_paged(pk, pv, pg, kp, vp, gp, table, seqlens, cu_seqlens=cu.cuda(), q=pq,
                                           inv_freq=f, return_k=True)
    q2, k2 = fixattn.fix_rotary(pq, pk, f, cu_seqlens=cu.cuda())
    assert torch.equal(qr, q2) and torch.equal(kr, k2)           # serving rotates as training does
    y, _ = fixattn.fix_attn_fwd(qr, kr, pv, pg, on["w"], cu.cuda(), cu, y_dtype=torch.float32, save=False)
    rows = {b: [y[0, int(cu[b]) + prompts[b] - 1]] for b in range(B)}
    for i in range(steps):
        seqlens += 1
        at = [(b, prompts[b] + i) for b in range(B)]
        new = {x: torch.stack([on[x][b, t] for b, t in at])[:, None].contiguous() for x in ("q", "k", "v", "g")}
        qr, _ = fixattn.fix_attn_append_paged(new["k"], new["v"], new["g"], kp, vp, gp, table, seqlens, q=new["q"],
                                              inv_freq=f)
        y = fixattn.fix_attn_decode_paged(qr[:, 0], kp, vp, gp, table, seqlens, on["w"], y_dtype=torch.float32)
        for b in range(B):
            rows[b].append(y[b])
    for b in range(B):
        L = prompts[b] + steps
        qf, kf = (rotate_ref(case[x][b, :L], range(L), inv_freq(D))[0].to(bf16)[None] for x in ("q", "k"))
        ref = fix_ref.forward(qf, kf, case["v"][b:b + 1, :L], case["g"][b:b + 1, :L], case["w"])["y"][0]
        for i, got in enumerate(rows[b]):
            want = torch.as_tensor(ref[prompts[b] - 1 + i])
            # the rotated q and k may round to other bf16 neighbours than the reference's: 5e-3 is the
            # forward's own bar
            assert float((got.double().cpu() - want).norm() / want.norm()) <= 5e-3, (b, i)


def _step(st):
    q, _ = fixattn.fix_attn_append_paged(st["k"], st["v"], st["g"], *st["pages"], st["table"], st["seqlens"],
                                         q=st["q"], inv_freq=st["f"])
    return fixattn.fix_attn_decode_paged(q[:, 0], *st["pages"], st["table"], st["seqlens"], st["w"],
                                         y_dtype=torch.float32)


def _step_state(lens, seed, Hq=8, Hkv=2, D=128, page=16, cols=64):
    c = Cache(lens, Hkv, D, D, page, seed=seed, cols=cols, spare=len(lens) * 12)
    used = set(c.table[c.table >= 0].tolist())
    spare = [i for i in range(c.k.shape[0]) if i not in used]
    for b in range(len(lens)):                                   # pages for tokens to come
        for col in range(-(-lens[b] // page), -(-lens[b] // page) + 12):
            c.table[b, col] = spare.pop()
    kp, vp, gp, table, seqlens = c.cuda()
    gen = torch.Generator().manual_seed(seed + 5)
    B = len(lens)
    st = {x: torch.randn(B, 1, h, D, generator=gen).to(bf16).cuda() for x, h in (("q", Hq), ("k", Hkv), ("v", Hkv))}
    st |= dict(g=(-torch.rand(B, 1, Hkv, D, generator=gen)).cuda(), pages=(kp, vp, gp), table=table,
               seqlens=seqlens, f=inv_freq(D).cuda(), w=torch.ones(D, dtype=bf16).cuda())
    return st


@pytest.mark.gpu
def test_captured_step_replays_with_other_lengths(cuda_lib):
    """One captured step (append and decode), replayed while lengths and
    inputs change in place, gives the eager calls' bits; a fixed-size batch
    carries a padding row."""
    st = _step_state([1, 200, 0, 47], 41)
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        _step(st)
    torch.cuda.current_stream().wait_stream(warm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = _step(st)
    gen = torch.Generator().manual_seed(3)
    for add in ([1, 1, 0, 1], [3, 150, 0, 9], [90, 0, 5, 1], [0, 0, -5, 0]):
        st["seqlens"] += torch.tensor(add, dtype=torch.int32).cuda()
        # tokens that were skipped in between: fill their slots
        for x in st["pages"]:
            x.copy_(torch.nan_to_num(x, nan=0.0))
        for name in ("q", "k", "v"):
            st[name].copy_(torch.randn(st[name].shape, generator=gen).to(bf16))
        graph.replay()
        got, pages = y.clone(), [x.clone() for x in st["pages"]]
        want = _step(st)
        assert torch.equal(got, want)
        assert all(torch.equal(a, b) for a, b in zip(pages, st["pages"]))
        assert bool((st["seqlens"] > 0).eq(got.flatten(1).any(1)).all())


@pytest.mark.gpu
def test_two_streams_at_once_and_given_workspace(cuda_lib):
    a, b = _step_state([700, 3, 512], 51), _step_state([31, 650], 52)
    for s in (a, b):
        for x in s["pages"]:
            x.copy_(torch.nan_to_num(x, nan=0.0))
    wa, wb = _step(a), _step(b)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(20):
        with torch.cuda.stream(sa):
            ya = _step(a)
        with torch.cuda.stream(sb):
            yb = _step(b)
        outs.append((ya, yb))
    torch.cuda.synchronize()
    assert all(torch.equal(x, wa) and torch.equal(y, wb) for x, y in outs)
    # the stream argument, a kept workspace and a given output
    q = a["q"][:, 0].contiguous()
    want = fixattn.fix_attn_decode_paged(q, *a["pages"], a["table"], a["seqlens"], a["w"])
    ws = fixattn.fix_attn_decode_paged_workspace(q, *a["pages"], a["table"], a["seqlens"])
    ws.fill_(255)
    out = torch.empty_like(want)
    sa.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        out.fill_(NAN)
        sa.wait_stream(torch.cuda.current_stream())
        got = fixattn.fix_attn_decode_paged(q, *a["pages"], a["table"], a["seqlens"], a["w"], workspace=ws, out=out,
                                            stream=sa)
        sa.synchronize()
        assert got is out and torch.equal(got, want)


@pytest.mark.gpu
def test_shared_pages_of_a_common_prefix(cuda_lib):
    """Two sequences whose tables name the same pages for their prefix."""
    c = Cache([64, 64], 2, 64, 64, 16, seed=61)
    c.table[1, :3] = c.table[0, :3]
    c.tok[1] = tuple(torch.cat((x[:48], y[48:])) for x, y in zip(c.tok[0], c.tok[1]))
    q, w, _ = decode_inputs(2, 4, 64, 64, 62)
    y = fixattn.fix_attn_decode_paged(q.cuda(), *c.cuda(), w.cuda(), y_dtype=torch.float32)
    check_decode(y, c, q, w, None)


@pytest.mark.gpu
def test_python_refusals_on_the_gpu(cuda_lib):
    c = Cache([20, 5], 2, 64, 64, 16)
    kp, vp, gp, table, seqlens = c.cuda()
    q = torch.zeros(2, 4, 64, dtype=bf16, device="cuda")
    w = torch.ones(64, dtype=bf16, device="cuda")
    x = torch.zeros(2, 1, 2, 64, dtype=bf16, device="cuda")
    f = inv_freq(64).cuda()
    ok = (q, kp, vp, gp, table, seqlens, w)

    def bad(i, t, exc=ValueError):
        with pytest.raises(exc):
            fixattn.fix_attn_decode_paged(*ok[:i], t, *ok[i + 1:])

    bad(0, q.float()); bad(0, q[:1]); bad(0, q.cpu()); bad(0, q.transpose(0, 1)); bad(0, None, TypeError)
    bad(0, torch.zeros(2, 4, 32, dtype=bf16, device="cuda"))
    bad(1, kp.float()); bad(1, kp.transpose(1, 2)); bad(2, vp[:-1]); bad(3, gp[..., :8]); bad(3, gp.to(bf16))
    bad(4, table.long()); bad(4, table.t()); bad(4, table[:1]); bad(4, table.cpu())
    bad(5, seqlens.long()); bad(5, seqlens[:1]); bad(6, None); bad(6, w.float()); bad(6, w[:32])
    for kw in (dict(o_gate=q.float()), dict(out=q[:1]), dict(y_dtype=torch.float16), dict(workspace=w),
               dict(status=torch.zeros(2, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            fixattn.fix_attn_decode_paged(*ok, **kw)
    with pytest.raises(fixattn.FixStatusError, match="WORKSPACE"):
        fixattn.fix_attn_decode_paged(*ok, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    pages = (kp, vp, gp, table, seqlens)
    for args, kw in (((x, x, gp), {}), ((x, x[..., :32], x.float()), {}), ((x, x, x.float()[..., 0]), {}),
                     ((x, x, x.float()), dict(q=q[:, None])), ((x, x, x.float()), dict(return_k=True)),
                     ((x, x, x.float()), dict(inv_freq=f[:12])), ((x, x, x.float()), dict(inv_freq=f.double())),
                     ((x, x, x.float()), dict(cu_seqlens=torch.tensor([0, 1, 2]).cuda())),
                     ((x.transpose(0, 1), x, x.float()), {})):
        with pytest.raises(ValueError):
            fixattn.fix_attn_append_paged(*args, *pages, **kw)
    for args, kw in (((x.float(), x, f), {}), ((x, x[:1], f), {}), ((x, x, f[None]), {}), ((x[0], x, f), {}),
                     ((x, x, f), dict(positions=torch.zeros(2, 1).cuda())), ((x, x, f), dict(out=(x, None))),
                     ((x, x, f), dict(cu_seqlens=torch.tensor([0, 2]).cuda()))):
        with pytest.raises(ValueError):
            fixattn.fix_attn_rotary(*args, **kw)
    with pytest.raises(fixattn.FixStatusError, match="HEAD_DIM"):
        y = torch.zeros(1, 1, 1, 96, dtype=bf16, device="cuda")
        fixattn.fix_attn_rotary(y, y, f)


@pytest.mark.gpu
def test_decode_paged_all_nan(cuda_lib):
    """NaN in every key, or in one value, of a sequence reaches its rows (as
    whole rows after the norm), and no other sequence's."""
    c = Cache([1, 20, 30, 9], 2, 64, 64, 16, seed=3)
    q, w, _ = decode_inputs(4, 4, 64, 64, 4)
    c.k[int(c.table[0, 0]), 0] = NAN
    for i in range(20):
        c.k[int(c.table[1, i // 16]), i % 16, 1] = NAN            # kv head 1: q heads 2, 3
    c.v[int(c.table[2, 0]), 5, 0, 7] = NAN                        # kv head 0: q heads 0, 1
    y = fixattn.fix_attn_decode_paged(q.cuda(), *c.cuda(), w.cuda(), y_dtype=torch.float32).cpu()
    nan = torch.isnan(y)
    assert bool(nan[0].all()) and bool(nan[1, 2:].all()) and not nan[1, :2].any()
    assert bool(nan[2, :2].all()) and not nan[2, 2:].any() and not nan[3].any()
    check = decode_ref(q[3], *c.tok[3], w, None, 64 ** -0.5, 1e-6, True)
    assert float((y[3] - check).norm() / check.norm()) <= F32_ROW


@pytest.mark.gpu
def test_rotary_gradient_as_autograd_calls_it(cuda_lib):
    """Gradients that are views off the 16-byte boundary, leaves that are
    broadcast, a second derivative, inputs changed before the backward, and a
    captured forward and backward."""
    gen = torch.Generator().manual_seed(9)
    B, T, H, D = 2, 6, 2, 32
    mk = lambda *s: torch.randn(*s, generator=gen).to(bf16)  # noqa: E731
    q, k, f = mk(B, T, H, D), mk(B, T, H, D), inv_freq(D)
    pos = [t for _ in range(B) for t in range(T)]
    ql, kl = q.cuda().requires_grad_(True), k.cuda().requires_grad_(True)
    fd = f.cuda()
    flat = mk(B * T * H * D + 1).cuda()
    off = flat[1:].view(B, T, H, D)                              # 2 bytes off
    gq, gk = torch.autograd.grad(fixattn.fix_rotary(ql, kl, fd), (ql, kl), (off, off))
    check_rotated(gq, off.cpu(), pos, f, False, True)
    check_rotated(gk, off.cpu(), pos, f, False, True)
    # one head's keys for all heads: the gradient is the sum over the copies
    one = mk(B, T, 1, D)
    ol = one.cuda().requires_grad_(True)
    dk = mk(B, T, H, D)
    _, kr = fixattn.fix_rotary(ql, ol.expand(B, T, H, D).contiguous(), fd)
    go, = torch.autograd.grad(kr, ol, dk.cuda())
    ref, mag = rotate_ref(dk.flatten(0, 1), pos, f, inverse=True)
    err = (go.double().cpu().flatten(0, 1) - ref.sum(1, keepdim=True)).abs()
    # a rounding of each summand and one of the sum
    bar = BF16 * (ref.abs().sum(1, keepdim=True) + ref.sum(1, keepdim=True).abs()) + 1e-6 * mag.sum(1, keepdim=True)
    assert bool((err <= bar).all())
    # the gradient is linear in the incoming one, with the rotation itself as derivative
    d = mk(B, T, H, D).cuda().requires_grad_(True)
    g1, = torch.autograd.grad(fixattn.fix_rotary(ql, kl, fd)[0], ql, d, create_graph=True)
    g2, = torch.autograd.grad(g1, d, off)
    check_rotated(g2, off.cpu(), pos, f)
    # positions changed between forward and backward
    positions = torch.zeros(B, T, dtype=torch.int32, device="cuda")
    qr, kr = fixattn.fix_rotary(ql, kl, fd, positions=positions)
    positions += 1
    with pytest.raises(RuntimeError, match="modified"):
        torch.autograd.grad((qr, kr), (ql, kl), (off, off))
    # captured, with leaves of its own (PyTorch ties a leaf's accumulation to the stream of the oldest graph
    # of it that lives: as with any of its operations, the capture fails while an eager one is)
    ql, kl = q.cuda().requires_grad_(True), k.cuda().requires_grad_(True)
    dq = mk(B, T, H, D).cuda()

    def step():
        a, b = fixattn.fix_rotary(ql, kl, fd)
        return (a, b) + torch.autograd.grad((a, b), (ql, kl), (dq, dq))

    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = step()
    with torch.no_grad():
        ql.copy_(mk(B, T, H, D))
        dq.copy_(mk(B, T, H, D))
    graph.replay()
    want = step()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.gpu
def test_integer_arrays_at_any_offset_and_the_unused_first_gate(cuda_lib):
    """Lengths, tables and sequence starts that are slices of larger buffers;
    and the gate of a sequence's first token, which no decay uses, as NaN."""
    lens, new = [300, 41, 5000], [1, 0, 2]
    c = Cache(lens, 2, 64, 64, 16, seed=71, gate=lambda x: -1e-3 * x.abs())
    for b in range(3):
        c.g[int(c.table[b, 0]), 0] = NAN
    kp, vp, gp, table, seqlens = c.cuda()
    q, w, _ = decode_inputs(3, 6, 64, 64, 72)
    ints = torch.cat((torch.zeros(1, dtype=torch.int32).cuda(), seqlens))
    tab = torch.cat((torch.zeros(3, dtype=torch.int32).cuda(), table.flatten()))
    args = (kp, vp, gp, tab[3:].view(table.shape), ints[1:])
    y = fixattn.fix_attn_decode_paged(q.cuda(), *args, w.cuda(), y_dtype=torch.float32)
    check_decode(y, c, q, w, None)
    cu = torch.tensor([7, 0, 1, 1, 3], dtype=torch.int64).cuda()[1:]
    f = torch.cat((torch.zeros(1), inv_freq(64))).cuda()[1:]
    x = torch.randn(1, 3, 2, 64, generator=torch.Generator().manual_seed(5)).to(bf16).cuda()
    fixattn.fix_attn_append_paged(x, x, x.float(), *args, cu_seqlens=cu, inv_freq=f)
    pos = [lens[0] - 1, lens[2] - 2, lens[2] - 1]
    got = torch.stack([kp[int(table[b, p // 16]), p % 16] for b, p in zip((0, 2, 2), pos)])
    check_rotated(got, x.cpu(), pos, inv_freq(64))


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,hi,scalar", [(300, 32, 2, 300, False), (300, 20, 2, 300, True),
                                                (600, 20, 4, 80, False)])
def test_decode_paged_many_rows_to_join(cuda_lib, B, Hq, Hkv, hi, scalar):
    """Thousands of (sequence, q head) rows whose pieces are joined, with fewer
    and with more units than the split has workers."""
    gen = torch.Generator().manual_seed(B + Hq)
    lens = torch.randint(0, hi, (B,), generator=gen).tolist()
    c = Cache(lens, Hkv, 32, 32, 16, seed=15, scalar=scalar)
    q, w, z = decode_inputs(B, Hq, 32, 32, 16, True)
    for norm in (True, False):
        y = fixattn.fix_attn_decode_paged(q.cuda(), *c.cuda(), w.cuda(), y_dtype=torch.float32, o_gate=z.cuda(),
                                          o_norm=norm)
        check_decode(y, c, q, w, z, norm=norm, rows=list(range(0, B, 23)) + [B - 1])


@pytest.mark.gpu
@pytest.mark.parametrize("between", ["copy", "clear", "other stream", "nothing"])
def test_captured_behind_copies_and_forks(cuda_lib, between):
    """The calls' kernels are launched to overlap the end of the kernel before
    them; in a graph they may follow a memory copy, a clear or a join of two
    streams just as well, and see what those wrote."""
    st = _step_state([30, 77], 81)
    for x in st["pages"]:
        x.copy_(torch.nan_to_num(x, nan=0.0))
    src = {n: st[n].clone() for n in ("k", "seqlens")}
    side, main = torch.cuda.Stream(), torch.cuda.Stream()

    def step():
        if between == "copy":
            st["seqlens"].copy_(src["seqlens"])
        elif between == "clear":
            st["k"].zero_()
        elif between == "other stream":
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                st["k"].copy_(src["k"])
            torch.cuda.current_stream().wait_stream(side)
        q, _ = fixattn.fix_attn_append_paged(st["k"], st["v"], st["g"], *st["pages"], st["table"], st["seqlens"],
                                             q=st["q"], inv_freq=st["f"])
        if between == "copy":
            st["seqlens"].copy_(src["seqlens"])
        elif between == "clear":
            src["seqlens"].zero_()
        return fixattn.fix_attn_decode_paged(q[:, 0], *st["pages"], st["table"], st["seqlens"], st["w"],
                                             y_dtype=torch.float32)

    main.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(main):
        want = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        y = step()
    for _ in range(3):
        y.fill_(NAN)
        if between == "other stream":
            st["k"].fill_(NAN)
        if between == "copy":
            st["seqlens"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
