"""The selection scans' rings of bulk copies in freshly started processes, where a slot that is filled before it is
read shows (GPU only): every scan form as a process's first call, against scores computed from the same plane."""
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
