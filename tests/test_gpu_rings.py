"""What the order of asynchronous work could break (GPU only): the selection scans' rings of bulk copies in freshly
started processes, where a slot that is filled before it is read shows, and reads that rest on a predecessor's wait."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

CODE = """
import sys, torch, sparse_attention_decode_loki_b200 as loki
form = sys.argv[1]
g = torch.Generator().manual_seed(17)
B, H, S, D, d, k, page = (16, 40, 4096, 128, 32, 64, 64) if form in ("paged8", "plane", "step") else (2 if form == "cluster" else 1, 8, 8000, 128, 32, 64, 80)
dt = torch.bfloat16
q = torch.randn(B, H, D, generator=g).cuda().to(dt)
P = torch.linalg.qr(torch.randn(H, D, D, generator=g))[0].contiguous().cuda()
gpu = torch.Generator(device="cuda").manual_seed(18)
lo = torch.randn(B, H, S, d, generator=gpu, device="cuda").to(dt)
if form == "paged8":
    n = B * S // page
    perm = torch.randperm(n, generator=g).cuda()
    bt = perm.to(torch.int32).view(B, S // page).contiguous()
    pages = torch.empty(n, H, page, d, dtype=dt, device="cuda")
    pages[perm] = lo.view(B, H, S // page, page, d).transpose(1, 2).reshape(n, H, page, d)
    c8 = torch.zeros(n, H, page, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    sc = torch.ones(n, H, page // 16, device="cuda")
    lens = torch.full((B,), S, dtype=torch.int32, device="cuda")
    _, idx = loki.loki_decode_attention_paged_q8(q, c8, c8, sc, sc, pages, P, bt, lens, d, k)
else:
    K = torch.zeros(B, H, S, D, dtype=dt, device="cuda")
    if form == "step":
        new = torch.randn(B, H, 1, D, generator=g).cuda().to(dt)
        _, idx = loki.loki_decode_step(q, new, new, P, K, K.clone(), S - 1, d, k, Kt_lo=lo)
    elif form == "fused":
        _, idx = loki.loki_decode_attention_fused(q, K, K, lo, P, S, d, k)
    else:
        _, idx = loki.loki_decode_attention_plane(q, K, K, lo, P, S, d, k)
torch.cuda.synchronize()
assert loki.loki_device_error(reset=True) == 0
qr = torch.einsum("bhd,hdc->bhc", q.double(), P.double())[..., :d]
score = torch.einsum("bhc,bhsc->bhs", qr, lo.double())
# fp32: D products of the rotated query, d of the score
bound = ((D + d + 8) * 2.0 ** -24 * q.double().abs().sum(-1, keepdim=True) * P.abs().max() * lo.double().abs().sum(-1).amax(-1, keepdim=True))
chosen = torch.zeros_like(score, dtype=torch.bool).scatter_(2, idx.long(), True)
assert bool((chosen.sum(-1) == k).all())
worst = torch.where(chosen, score, score.new_tensor(float("inf"))).amin(-1, keepdim=True)
assert bool(((score <= worst + 2 * bound) | chosen).all())
"""


@pytest.mark.parametrize("form", ["paged8", "plane", "step", "fused", "cluster"])
def test_first_selections_of_new_processes(cuda, form):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    jobs = [subprocess.Popen([sys.executable, "-c", CODE, form], cwd=root) for _ in range(4)]
    assert [j.wait(timeout=300) for j in jobs] == [0] * 4


@pytest.fixture(scope="module")
def loki(cuda):
    import sparse_attention_decode_loki_b200 as m
    return m


@pytest.mark.parametrize("T,H,q8", [(17, 1, False), (17, 1, True), (100, 2, True), (300, 8, False)])
def test_values_and_queries_rewritten_in_place(loki, cuda, T, H, q8):
    """A long append's stream of values and queries does not wait for what came before the keys' kernel, which
    did: inputs, positions and angles that every SM has read just before, rewritten in place, call after call."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=g, device=cuda).to(torch.bfloat16)  # noqa: E731
    n = 8 * T + 64
    K, V, q, q_out = rnd(1, H, T, 128), rnd(1, H, T, 128), rnd(1, 4 * H, T, 128), rnd(1, 4 * H, T, 128)
    Kp, Vp = (torch.zeros(1, H, (n + 15) // 16 * 16, 128, dtype=torch.bfloat16, device=cuda) for _ in range(2))
    tab = loki.loki_rope_table(n, 128, device=cuda)
    bt, pos = torch.zeros(1, 1, dtype=torch.int32, device=cuda), torch.zeros(1, dtype=torch.int32, device=cuda)
    if q8:
        Kp, Vp = (t.to(torch.float8_e4m3fn) for t in (Kp, Vp))
        ks, vs = (torch.ones(1, H, Kp.shape[2] // 16, device=cuda) for _ in range(2))
    wrong = torch.zeros((), dtype=torch.int64, device=cuda)
    at = torch.arange(T, device=cuda)
    many = torch.zeros(148 * 16, 1, device=cuda)
    for i in range(200):
        for t in (V, q, tab):  # every SM reads all of them
            (many + t.view(-1)[:2048].float()).sum()
        V.neg_()
        q.mul_(-1.0)
        tab.neg_()  # (cos and sin change sign together: the turned queries too)
        pos.fill_(16 * (i % 7))
        a = (K, V, None, Kp, Vp)
        if q8:
            loki.loki_append_keys_paged_q8(*a, ks, vs, bt, pos, rope_table=tab, q=q, q_out=q_out)
            got = Vp.view(torch.uint8)[0, :, 16 * (i % 7) + at].view(torch.float8_e4m3fn).float()
            err = (torch.sign(got) * torch.sign(V[0].float()) < 0).sum()
        else:
            loki.loki_append_keys_paged_rope(*a, bt, pos, rope_table=tab, q=q, q_out=q_out)
            err = (Vp[0, :, 16 * (i % 7) + at] != V[0]).sum()
        c, s = (t[None] for t in tab[16 * (i % 7) + at].chunk(2, -1))
        lo, hi = q[0].float().chunk(2, -1)
        want = torch.cat([lo * c - hi * s, lo * s + hi * c], -1)
        off = (q_out[0].float() - want).abs() > 2.0 ** -8 * (want.abs() + 2.0 ** -21 * 8) + 2.0 ** -21 * 8
        wrong += err + off.sum()
    assert int(wrong) == 0 and loki.loki_device_error(reset=True) == 0


def test_lengths_rewritten_in_place(loki, cuda):
    """The two-kernel attention's merge reads the lengths before it waits: lengths that every SM has read just
    before, rewritten in place, call after call."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(6)
    n, page = 6000, 16
    K8, V8 = ((torch.randn(n // page, 1, page, 128, generator=g, device=cuda) * 80).to(torch.float8_e4m3fn) for _ in range(2))
    sc = torch.full((n // page, 1, 1), 2.0 ** -6, device=cuda)
    bt = torch.full((2, 16000), -1, dtype=torch.int32, device=cuda)
    bt[:, : n // page] = torch.arange(n // page, device=cuda)
    q = torch.randn(2, 4, 128, generator=g, device=cuda)
    lens = [[0, 6000], [6000, 17], [33, 0], [1, 5000], [2500, 2500], [0, 0]]
    want = [loki.dense_decode_attention_paged_q8(q, K8, V8, sc, sc, bt, torch.tensor(x, dtype=torch.int32, device=cuda)).clone()
            for x in lens]
    sl, rows = torch.zeros(2, dtype=torch.int32, device=cuda), torch.tensor(lens, dtype=torch.int32, device=cuda)
    many, wrong = torch.zeros(148 * 2048, 1, device=cuda), torch.zeros((), dtype=torch.int64, device=cuda)
    out = torch.empty_like(q)
    for i in range(300):
        (many + sl.float()).sum()
        sl.copy_(rows[i % 6])
        loki.dense_decode_attention_paged_q8(q, K8, V8, sc, sc, bt, sl, out=out)
        wrong += (out != want[i % 6]).sum()
    assert int(wrong) == 0 and loki.loki_device_error(reset=True) == 0
