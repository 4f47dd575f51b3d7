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
