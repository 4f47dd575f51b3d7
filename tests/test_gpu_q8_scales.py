"""Scales of 8-bit pages over the whole range that the contract allows (any finite scale >= 0, not only the
powers of two that the appends write), against the fp64 restatement in tests/q8_ref.py (GPU only)."""
from __future__ import annotations

import math

import numpy as np
import pytest

from tests import q8_ref
from tests.test_gpu_q8_attention import pool, rows_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def loki(cuda):
    import sparse_attention_decode_loki_b200 as m
    return m


def attentions(loki, torch, q, K8, V8, ks, vs, bt, sl, scale=0.0):
    """The same tokens through the dense attention and through the selected one, in the form that a table of
    just their pages (a list of just them) takes and in the form of a long table (list): fp32 outputs."""
    page, n = K8.shape[2], int(sl.max())
    short = bt[:, : -(-n // page)].contiguous()
    wide = torch.full((bt.shape[0], (1 << 19) // page), -1, dtype=torch.int32, device=bt.device)
    wide[:, : short.shape[1]] = short
    idx = torch.arange(n, dtype=torch.int32, device=bt.device).expand(*q.shape[:2], n).contiguous()
    far = torch.full((*q.shape[:2], 400000), -1, dtype=torch.int32, device=bt.device)
    far[..., :n] = idx
    pages = (K8, V8, ks, vs)
    yield "dense, clusters", loki.dense_decode_attention_paged_q8(q, *pages, short, sl, scale=scale)
    yield "dense, two kernels", loki.dense_decode_attention_paged_q8(q, *pages, wide, sl, scale=scale)
    for tag, i in (("selected, clusters", idx), ("selected, two kernels", far)):
        yield tag, loki.loki_sparse_attention_paged_q8(q, *pages, short, sl, i, scale=scale, dtype=torch.float32)


def compare(loki, torch, q, K8, V8, ks, vs, bt, sl, block, scale=0.0):
    page, n, H = K8.shape[2], int(sl[0]), K8.shape[1]
    K, V = rows_of(K8, ks, bt, 0, n, page, block), rows_of(V8, vs, bt, 0, n, page, block)
    for tag, out in attentions(loki, torch, q, K8, V8, ks, vs, bt, sl, scale):
        o, qn = out[0].double().cpu().numpy(), q[0].double().cpu().numpy()
        assert np.all(np.isfinite(o)), tag
        for h in range(q.shape[1]):
            Kh, Vh, sc = K[h * H // q.shape[1]], V[h * H // q.shape[1]], scale or q.shape[2] ** -0.5
            ref = q8_ref.attend(qn[h], Kh, Vh, sc)
            tol = q8_ref.attend_tol(qn[h], Kh, Vh, sc, ref, 2.0 ** -24)
            assert np.all(np.abs(o[h] - ref) <= tol + 2.0 ** -149), (tag, h, np.abs(o[h] - ref).max(), tol.max())
    assert loki.loki_device_error(reset=True) == 0


@pytest.mark.parametrize("n,block", [(1, 16), (100, 16), (900, 32)])
def test_scales_that_are_no_powers_of_two(loki, cuda, n, block):
    """Any finite scale from zero on, block by block."""
    import torch
    K8, V8, ks, vs, bt, sl = pool(torch, cuda, 2, 128, 64, block, [n], -(-n // 64) + 1, 61)
    g = torch.Generator().manual_seed(62)
    for t, lo, hi in ((ks, -14, -7), (vs, -30, 20)):
        t.copy_(torch.exp2(torch.rand(t.shape, generator=g) * (hi - lo) + lo))
        t.view(-1)[::7] = 0.0
    q = torch.randn(1, 8, 128, generator=g).to(cuda)
    compare(loki, torch, q, K8, V8, ks, vs, bt, sl, block)


def test_zero_values_under_a_score_far_above_large_ones(loki, cuda):
    """In every warp's run: tiles of large values, then tiles of zeros (least scale) whose score lies 144
    binades higher. The large values' share is some 2^-144 of the output."""
    import torch
    n, page = 4800, 16  # 300 tiles: several for each warp of a cluster too
    K8, V8, ks, vs, bt, sl = pool(torch, cuda, 1, 128, page, 16, [n], n // page, 63)
    p = bt[0].long()
    K8.view(torch.uint8).zero_()
    at = torch.arange(n // page, device=cuda)
    top = torch.where(at % 4 == 1, 144.0, torch.where(at % 4 == 3, 64.0, 0.0)).to(torch.float8_e4m3fn)
    K8.view(torch.uint8)[p, 0, :, 0] = top.view(torch.uint8)[:, None]
    ks.fill_(1.0)
    V8.view(torch.uint8)[p[at % 4 == 1]] = 0
    vs[p, 0, 0] = torch.where(at % 4 == 1, 2.0 ** -126, torch.where(at % 4 == 0, 2.0 ** 30, 2.0 ** -20))
    q = torch.zeros(1, 4, 128, device=cuda)
    q[..., 0] = 1.0
    compare(loki, torch, q, K8, V8, ks, vs, bt, sl, 16, scale=math.log(2.0))  # scores in binades


@pytest.mark.parametrize("s", [1.5 * 2.0 ** 127, 2.0 ** 126, 3e-33, 2.0 ** -108, 2.0 ** -120])
def test_values_near_the_ends_of_fp32(loki, cuda, s):
    """One token whose values lie near fp32's largest, and few whose values lie near its smallest: weights
    keep their bits relative to the largest value."""
    import torch
    n = 1 if s > 1 else 40
    K8, V8, ks, vs, bt, sl = pool(torch, cuda, 1, 128, 16, 16, [n], 3, 64)
    V8.copy_((torch.rand(V8.shape, generator=torch.Generator().manual_seed(65)) * 2 - 1).to(torch.float8_e4m3fn))
    vs.fill_(s)
    q = torch.randn(1, 4, 128, generator=torch.Generator().manual_seed(66)).to(cuda)
    compare(loki, torch, q * 0.1, K8, V8, ks, vs, bt, sl, 16)


def test_small_values_among_many_tokens(loki, cuda):
    """Values around 1e-33 of many tokens with the same score: the weights' sum is large, 2^-E is too."""
    import torch
    n = 20000
    K8, V8, ks, vs, bt, sl = pool(torch, cuda, 1, 128, 32, 32, [n], n // 32, 67)
    vs.fill_(2.0 ** -114)
    K8.view(torch.uint8).zero_()
    q = torch.randn(1, 4, 128, generator=torch.Generator().manual_seed(68)).to(cuda)
    compare(loki, torch, q, K8, V8, ks, vs, bt, sl, 32)


@pytest.mark.parametrize("qs,s", [(5e37, 1e-38), (1e-37, 5e34)])
def test_queries_and_keys_of_opposite_sizes(loki, cuda, qs, s):
    """Scores of ordinary size from queries near one end of fp32 and keys near the other."""
    import torch
    n = 300
    K8, V8, ks, vs, bt, sl = pool(torch, cuda, 2, 128, 32, 16, [n], 11, 69)
    ks.fill_(s)
    q = (torch.randn(1, 8, 128, generator=torch.Generator().manual_seed(70)) * qs).to(cuda)
    compare(loki, torch, q, K8, V8, ks, vs, bt, sl, 16)


@pytest.mark.parametrize("T", [1, 5, 40])
@pytest.mark.parametrize("basis", [False, True], ids=["noP", "P"])
@pytest.mark.parametrize("old", [0.0, 0.3, 0.0071, 1.9 * 2.0 ** 30, 1.7 * 2.0 ** 126, 3.0 * 2.0 ** -140])
def test_appends_behind_blocks_of_any_scale(loki, cuda, T, basis, old):
    """Older tokens of a block whose scale is no power of two: it stays, or its codes move to the new one."""
    import torch
    H, D, page, block, pos = 2, 128, 32, 16, 11
    g = torch.Generator().manual_seed(72)
    rnd = lambda *s: torch.randn(*s, generator=g).to(cuda)  # noqa: E731
    n = -(-(pos + T) // page)
    K, V = rnd(1, H, T, D), rnd(1, H, T, D)
    P = torch.linalg.qr(torch.randn(H, D, D, generator=g))[0].contiguous().to(cuda) if basis else None
    K8, V8 = ((rnd(n, H, page, D) * 80).to(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.full((n, H, page // block), old, device=cuda) for _ in range(2))
    bt = torch.arange(n, dtype=torch.int32, device=cuda)[None].contiguous()
    was = [t.double().cpu().numpy() for t in (K8, V8)]
    loki.loki_append_keys_paged_q8(K, V, P, K8, V8, ks, vs, bt, torch.tensor([pos], dtype=torch.int32, device=cuda))
    torch.cuda.synchronize()
    assert loki.loki_device_error(reset=True) == 0
    x = K.double().cpu().numpy()[0]
    p = None if P is None else P.double().cpu().numpy()
    rows = (x if p is None else np.einsum("htd,hdc->htc", x, p), V.double().cpu().numpy()[0])
    # fp32 keys: D products of 22-bit parts summed with the basis; the values are exact
    bound = (0.0 if p is None else (D + 4) * 2.0 ** -24 * np.abs(x).max() * np.abs(p).sum(1).max(), 0.0)
    old32 = float(np.float32(old))
    for codes, scales, before, x, b in zip((K8, V8), (ks, vs), was, rows, bound):
        got, sc = codes.double().cpu().numpy(), scales.double().cpu().numpy()
        for h in range(H):
            for a in range(0, pos + T, block):
                first, z = max(pos - a, 0) % block if a <= pos else 0, min(a + block, pos + T)
                y = x[h, a + first - pos:z - pos]
                c0 = before[a // page, h, a % page:a % page + block]
                want, s = q8_ref.append_block(c0, old32, y, first)
                assert sc[a // page, h, a % page // block] == s
                c = got[a // page, h, a % page:a % page + block]
                # the exact quotient moved by the bound and by the roundings of a reciprocal (or of the scales'
                # quotient) and of a product, 2^-23 of it: the code lies between the two ends' codes
                for part, exact, off in ((slice(0, first), c0[:first] * (old32 / s) if s > old32 else c0[:first], 0.0),
                                         (slice(first, first + len(y)), y / s, b / s)):
                    off = off + 2.0 ** -23 * np.abs(exact) * (1.0 + 2.0 ** 4 * (s > 2.0 ** 126))  # (subnormal reciprocals)
                    lo, hi = q8_ref.e4m3_round(exact - off), q8_ref.e4m3_round(exact + off)
                    assert np.all((c[part] >= lo) & (c[part] <= hi)), (h, a, part)
                assert np.array_equal(c[first + len(y):], c0[first + len(y):])
