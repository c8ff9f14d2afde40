"""The backward of ``fix_rotary`` while autograd holds its tensors in another
form: non-reentrant checkpoints, offload to the host, hooks of a program's own.
Only what the saved tensors unpack to is alive then, and only that may reach
the kernel."""
import ctypes

import pytest
import torch
from torch.utils.checkpoint import checkpoint

from gated_softmax_attention_fp32_b200 import fixattn

bf16 = torch.bfloat16


def freqs(rot, device="cpu"):
    return (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)).float()


# ------------------------------------------------------------------ addresses, with the library call replaced (CPU)
class _Recorder:
    """Stands in for the library: notes the addresses and sizes of each call and copies q and k over."""

    def __init__(self):
        self.calls = []

    def fix_attn_rotary(self, p, r, positions, q, qs, k, ks, q_out, k_out, inverse, stream):
        n = p.batch * p.seqlen * p.head_dim_k * 2
        ctypes.memmove(q_out, q, n * p.num_q_heads)
        ctypes.memmove(k_out, k, n * p.num_kv_heads)
        self.calls.append(dict(inv_freq=r.inv_freq, cu=p.cu_seqlens, positions=positions, inverse=inverse,
                               sizes=(p.batch, p.seqlen, p.num_q_heads, p.num_kv_heads, p.head_dim_k, p.num_seqs,
                                      r.rot_dim, r.interleaved)))
        return 0


@pytest.fixture
def recorder(monkeypatch):
    rec = _Recorder()
    monkeypatch.setattr(fixattn, "load", lambda: rec)
    monkeypatch.setattr(fixattn, "_cuda_index", lambda name, t: t.get_device())
    monkeypatch.setattr(fixattn, "_elsewhere", lambda index, stream: None)
    monkeypatch.setattr(fixattn, "_raw_stream", lambda index: 0)
    return rec


def _leaves():
    return (torch.randn(1, 6, 4, 32).to(bf16).requires_grad_(True),
            torch.randn(1, 6, 2, 32).to(bf16).requires_grad_(True))


@pytest.mark.parametrize("packed", [False, True])
def test_backward_takes_addresses_from_the_unpacked_tensors(recorder, packed):
    unpacked = []

    def unpack(t):
        unpacked.append(t.clone())
        return unpacked[-1]

    q, k = _leaves()
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t.clone(), unpack):
        qr, kr = fixattn.fix_rotary(q, k, freqs(16),
                                    cu_seqlens=torch.tensor([0, 2, 6]) if packed else None,
                                    positions=None if packed else torch.arange(6, dtype=torch.int32)[None],
                                    interleaved=True)
    torch.autograd.grad((qr, kr), (q, k), (torch.ones_like(qr), torch.ones_like(kr)))
    fwd, bwd = recorder.calls
    assert bwd["sizes"] == fwd["sizes"] and (fwd["inverse"], bwd["inverse"]) == (0, 1)
    live = [t.data_ptr() for t in unpacked]
    assert len(live) == 2
    assert [bwd["inv_freq"], bwd["cu"] if packed else bwd["positions"]] == live
    assert not (bwd["positions"] if packed else bwd["cu"])


def test_backward_under_a_checkpoint_uses_the_recomputed_tensors(recorder):
    made = []

    def block(q, k):
        made.append((freqs(32), torch.arange(6)[None].to(torch.int32)))
        return fixattn.fix_rotary(q, k, made[-1][0], positions=made[-1][1])

    q, k = _leaves()
    qr, kr = checkpoint(block, q, k, use_reentrant=False)
    torch.autograd.grad((qr, kr), (q, k), (torch.ones_like(qr), torch.ones_like(kr)))
    assert len(made) == 2
    bwd = [c for c in recorder.calls if c["inverse"]]
    assert len(bwd) == 1
    assert (bwd[0]["inv_freq"], bwd[0]["positions"]) == tuple(t.data_ptr() for t in made[1])


def test_what_a_hook_returns_is_checked(recorder):
    """A hook that gives back another type or shape must not reach the kernel."""
    for wrong in (lambda t: t.double(), lambda t: t[..., :-1], lambda t: t.repeat_interleave(2, -1)[..., ::2]):
        q, k = _leaves()
        with torch.autograd.graph.saved_tensors_hooks(lambda t: t.clone(), wrong):
            qr, kr = fixattn.fix_rotary(q, k, freqs(32), positions=torch.arange(6, dtype=torch.int32)[None])
        with pytest.raises(ValueError):
            torch.autograd.grad((qr, kr), (q, k), (torch.ones_like(qr), torch.ones_like(kr)))
    assert not any(c["inverse"] for c in recorder.calls)


# ------------------------------------------------------------------ gradients (GPU)
@pytest.mark.gpu
@pytest.mark.parametrize("how", ["checkpoint", "offload", "own hooks"])
@pytest.mark.parametrize("packed", [False, True])
def test_gradients_with_tensors_made_inside(cuda_lib, how, packed):
    """Frequencies, positions and sequence starts that only the block knows,
    with allocations of the same sizes between forward and backward: the
    gradients are those of the plain call, bit for bit."""
    gen = torch.Generator().manual_seed(1)
    N, Hq, Hkv, D = 500, 4, 2, 64
    mk = lambda h: torch.randn(1, N, h, D, generator=gen).to(bf16).cuda()  # noqa: E731
    q, k, dq, dk = mk(Hq), mk(Hkv), mk(Hq), mk(Hkv)
    q.requires_grad_(True)
    k.requires_grad_(True)

    def block(q, k):
        f = freqs(D, "cuda")
        if packed:
            cu = torch.tensor([0, 3, 3, 401, N]).cuda()
            return fixattn.fix_rotary(q, k, f, cu_seqlens=cu)
        positions = torch.arange(7, 7 + N, device="cuda")[None].to(torch.int32)
        return fixattn.fix_rotary(q, k, f, positions=positions)

    want = torch.autograd.grad(block(q, k), (q, k), (dq, dk))
    if how == "checkpoint":
        out = checkpoint(block, q, k, use_reentrant=False)
    elif how == "offload":
        with torch.autograd.graph.save_on_cpu():
            out = block(q, k)
    else:
        with torch.autograd.graph.saved_tensors_hooks(lambda t: t + 1, lambda t: t - 1):
            out = block(q, k)
    # the allocator hands the freed blocks out again, with other contents
    junk = [torch.full((n,), 3, dtype=t, device="cuda") for n, t in
            ((D // 2, torch.float32), (N, torch.int32), (5, torch.int64)) for _ in range(16)]
    got = torch.autograd.grad(out, (q, k), (dq, dk))
    if how == "own hooks":      # f + 1 - 1 is another float than f: the forms of the tensors are what is tested
        f1 = freqs(D, "cuda") + 1 - 1
        where = (dict(cu_seqlens=torch.tensor([0, 3, 3, 401, N]).cuda()) if packed else
                 dict(positions=torch.arange(7, 7 + N, device="cuda")[None].to(torch.int32)))
        want = fixattn.fix_attn_rotary(dq, dk, f1, inverse=True, **where)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    del junk
