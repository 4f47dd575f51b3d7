"""Attention over paged 8-bit caches against the fp64 restatement (GPU only):
dense_decode_attention_paged_q8, loki_sparse_attention_paged_q8 and the decode
loki_decode_attention_paged_q8, alone and behind the appends that fill the cache."""
from __future__ import annotations

import numpy as np
import pytest

from tests import q8_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def loki(cuda):
    import sparse_attention_decode_loki_b200 as m
    return m


def pool(torch, dev, H_kv, D, page, block, lens, max_pages, seed, spread=2, spare=2):
    """Random codes and scales; pages in use hold NaN codes behind their sequence's end, spare pages
    NaN codes and scales; the table is -1 (or a wild number) where a sequence has no page."""
    g = torch.Generator(device="cpu").manual_seed(seed)
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + spare
    order = torch.randperm(n_pages, generator=g).tolist()
    bt = torch.full((len(lens), max_pages), -1, dtype=torch.int32)
    bt[:, -1] = 1 << 30
    shape = (n_pages, H_kv, page, D)
    K = (torch.randn(shape, generator=g) * 80).to(torch.float8_e4m3fn).view(torch.uint8)
    V = (torch.randn(shape, generator=g) * 80).to(torch.float8_e4m3fn).view(torch.uint8)
    sc = [torch.exp2(torch.randint(-8 - spread, -7, (n_pages, H_kv, page // block), generator=g).float())
          for _ in range(2)]
    live = torch.zeros(n_pages, page, dtype=torch.bool)
    for b, n in enumerate(lens):
        for lp in range(need[b]):
            p = order.pop()
            bt[b, lp] = p
            live[p, : min(page, n - lp * page)] = True
    K = torch.where(live[:, None, :, None], K, torch.full_like(K, 0x7F))
    V = torch.where(live[:, None, :, None], V, torch.full_like(V, 0xFF))
    dead = ~live.view(n_pages, page // block, block).any(-1)
    for t in sc:
        t.masked_fill_(dead[:, None], float("nan"))
    f8 = lambda t: t.to(dev).contiguous().view(torch.float8_e4m3fn)  # noqa: E731
    return (f8(K), f8(V), sc[0].to(dev).contiguous(), sc[1].to(dev).contiguous(), bt.to(dev),
            torch.tensor(lens, dtype=torch.int32, device=dev))


def rows_of(K8, ks, bt, b, n, page, block):
    """The cached values [H_kv, n, D] of sequence b, fp64."""
    K, s, t = K8.double().cpu().numpy(), ks.double().cpu().numpy(), bt.cpu().numpy()
    j = np.arange(n)
    p, at = t[b, j // page], j % page
    return np.moveaxis(K[p, :, at] * s[p, :, at // block][..., None], 0, 1)


def check(out, q, K, V, scale, half_step, tag):
    ref = q8_ref.attend(q, K, V, scale)
    tol = q8_ref.attend_tol(q, K, V, scale, ref, half_step)
    assert np.all(np.abs(out - ref) <= tol + 1e-30), (tag, np.abs(out - ref).max(), tol.max())


CASES = [
    # H_kv, G, D, dtype, page, block, lens
    (1, 1, 128, "bf16", 16, 16, [1]),
    (2, 1, 128, "f32", 16, 16, [15, 16, 17, 0]),
    (3, 4, 128, "bf16", 32, 16, [100, 1, 513]),
    (2, 8, 128, "bf16", 64, 64, [64, 63, 65, 640]),
    (2, 3, 96, "bf16", 48, 16, [47, 200, 0, 1]),
    (1, 5, 96, "f32", 128, 32, [300, 129]),
    (4, 2, 128, "f32", 256, 128, [1000]),
    (1, 7, 128, "bf16", 128, 128, [4097, 2]),
    (8, 4, 128, "bf16", 64, 32, [5000, 31, 777]),
    (40, 1, 128, "bf16", 64, 16, [130] * 9),
    (2, 6, 96, "f32", 16, 16, [9, 8, 7, 6, 5, 4, 3, 2, 1, 0]),
    (1, 1, 128, "bf16", 32, 32, [20000]),
]


def ids(c):
    return "H%d-G%d-D%d-%s-p%d-blk%d-n%d" % (c[0], c[1], c[2], c[3], c[4], c[5], max(c[6]))


@pytest.mark.parametrize("case", CASES, ids=ids)
@pytest.mark.parametrize("scale", [0.0, 0.3])
def test_dense_q8_matches_fp64(loki, cuda, case, scale):
    import torch
    H, G, D, dtn, page, block, lens = case
    dt = torch.bfloat16 if dtn == "bf16" else torch.float32
    max_pages = max(1, -(-max(lens) // page)) + 1
    K8, V8, ks, vs, bt, sl = pool(torch, cuda, H, D, page, block, lens, max_pages, 21)
    q = torch.randn(len(lens), H * G, D, generator=torch.Generator().manual_seed(3)).to(cuda).to(dt)
    q[:, :, ::7] *= 5
    out = loki.dense_decode_attention_paged_q8(q, K8, V8, ks, vs, bt, sl, scale=scale)
    torch.cuda.synchronize()
    assert loki.loki_device_error(reset=True) == 0
    o, qn = out.double().cpu().numpy(), q.double().cpu().numpy()
    for b, n in enumerate(lens):
        K, V = rows_of(K8, ks, bt, b, n, page, block), rows_of(V8, vs, bt, b, n, page, block)
        for h in range(H * G):
            check(o[b, h], qn[b, h], K[h // G], V[h // G], scale or D ** -0.5,
                  torch.finfo(dt).eps / 2, (b, h))


@pytest.mark.parametrize("case", CASES, ids=ids)
@pytest.mark.parametrize("frac", [1.0, 0.2])
def test_sparse_q8_matches_fp64(loki, cuda, case, frac):
    import torch
    H, G, D, dtn, page, block, lens = case
    dt = torch.bfloat16 if dtn == "bf16" else torch.float32
    max_pages = max(1, -(-max(lens) // page)) + 1
    K8, V8, ks, vs, bt, sl = pool(torch, cuda, H, D, page, block, lens, max_pages, 22)
    q = torch.randn(len(lens), H * G, D, generator=torch.Generator().manual_seed(4)).to(cuda)
    k = max(1, int(max(lens) * frac))
    rng = np.random.default_rng(5)
    idx = np.full((len(lens), H * G, k), -1, np.int32)
    for b, n in enumerate(lens):
        for h in range(H * G):
            m = min(k, n)
            idx[b, h, :m] = np.sort(rng.permutation(n)[:m])
            if h % 3 == 1 and k > 2:  # skipped entries among the valid ones
                idx[b, h, rng.integers(0, k, 2)] = [-5, n]
            if h % 3 == 2 and k > 2 and n:  # the same token twice, out of order
                idx[b, h, rng.integers(0, k, 2)] = n - 1
            if h == H * G - 1 and b == 0 and H * G > 1:  # a row with nothing to attend to
                idx[b, h] = -1
    out = loki.loki_sparse_attention_paged_q8(q, K8, V8, ks, vs, bt, sl, torch.from_numpy(idx).to(cuda), dtype=dt)
    torch.cuda.synchronize()
    assert loki.loki_device_error(reset=True) == 0
    o, qn = out.double().cpu().numpy(), q.double().cpu().numpy()
    for b, n in enumerate(lens):
        K, V = rows_of(K8, ks, bt, b, n, page, block), rows_of(V8, vs, bt, b, n, page, block)
        for h in range(H * G):
            i = idx[b, h]
            i = i[(i >= 0) & (i < n)]
            check(o[b, h], qn[b, h], K[h // G][i], V[h // G][i], D ** -0.5, torch.finfo(dt).eps / 2, (b, h))


def test_scales_far_apart_and_zero_blocks(loki, cuda):
    """Blocks whose scales differ by many binades, and the least scale of an all-zero block, keep the
    weighted sum exact to fp32 relative to the values that count."""
    import torch
    K8, V8, ks, vs, bt, sl = pool(torch, cuda, 2, 128, 64, 16, [640], 10, 23)
    V8.view(torch.uint8)[bt[0, 0].item(), :, :32] = 0
    vs[bt[0, 0].item(), :, :2] = 2.0 ** -126
    vs[bt[0, 3].item(), :, 1] = 2.0 ** 20
    vs[bt[0, 7].item(), :, 2] = 2.0 ** -60
    ks[bt[0, 3].item(), :, 1] = 2.0 ** -20
    q = torch.randn(1, 4, 128, generator=torch.Generator().manual_seed(6)).to(cuda)
    out = loki.dense_decode_attention_paged_q8(q, K8, V8, ks, vs, bt, sl)
    K, V = rows_of(K8, ks, bt, 0, 640, 64, 16), rows_of(V8, vs, bt, 0, 640, 64, 16)
    for h in range(4):
        check(out[0, h].double().cpu().numpy(), q[0, h].double().cpu().numpy(), K[h // 2], V[h // 2],
              128 ** -0.5, 2.0 ** -24, h)
    # every value zero: zeros, whatever the scales
    V8.view(torch.uint8).zero_()
    vs.fill_(2.0 ** -126)
    out = loki.dense_decode_attention_paged_q8(q, K8, V8, ks, vs, bt, sl)
    assert torch.all(out == 0)


def test_one_huge_score_and_all_equal_scores(loki, cuda):
    import torch
    K8, V8, ks, vs, bt, sl = pool(torch, cuda, 1, 128, 32, 32, [333], 12, 24)
    V = rows_of(V8, vs, bt, 0, 333, 32, 32)
    K = rows_of(K8, ks, bt, 0, 333, 32, 32)
    q = torch.from_numpy(K[:, 123] * 1e4).float().to(cuda)[None]
    out = loki.dense_decode_attention_paged_q8(q, K8, V8, ks, vs, bt, sl)
    # the winner takes all: the next score is thousands below in the exponent
    best = np.argmax(K[0] @ K[0, 123])
    assert np.array_equal(out[0, 0].double().cpu().numpy(), V[0, best])
    out = loki.dense_decode_attention_paged_q8(torch.zeros_like(q), K8, V8, ks, vs, bt, sl)
    check(out[0, 0].double().cpu().numpy(), np.zeros(128), K[0], V[0], 128 ** -0.5, 2.0 ** -24, "mean")


def test_bad_pages_are_skipped_and_flagged(loki, cuda):
    import torch
    K8, V8, ks, vs, bt, sl = pool(torch, cuda, 2, 128, 32, 16, [100, 50], 5, 25)
    q = torch.randn(2, 4, 128, generator=torch.Generator().manual_seed(7)).to(cuda)
    K, V = rows_of(K8, ks, bt, 0, 100, 32, 16), rows_of(V8, vs, bt, 0, 100, 32, 16)
    bt[0, 1] = -3
    keep = np.r_[0:32, 64:100]
    out = loki.dense_decode_attention_paged_q8(q, K8, V8, ks, vs, bt, sl)
    torch.cuda.synchronize()
    assert loki.loki_device_error(reset=True) == 2
    for h in range(4):
        check(out[0, h].double().cpu().numpy(), q[0, h].double().cpu().numpy(), K[h // 2][keep],
              V[h // 2][keep], 128 ** -0.5, 2.0 ** -24, h)
    bt[0, :] = K8.shape[0]  # no page of sequence 0 left: zeros; the other sequence is not touched by it
    idx = torch.arange(50, dtype=torch.int32, device=cuda).expand(2, 4, 50).contiguous()
    for f in (lambda: loki.dense_decode_attention_paged_q8(q, K8, V8, ks, vs, bt, sl),
              lambda: loki.loki_sparse_attention_paged_q8(q, K8, V8, ks, vs, bt, sl, idx, dtype=torch.float32)):
        o = f()
        torch.cuda.synchronize()
        assert loki.loki_device_error(reset=True) == 2
        assert torch.all(o[0] == 0) and torch.all(torch.isfinite(o[1])) and torch.any(o[1] != 0)


def test_lengths_are_clamped(loki, cuda):
    import torch
    K8, V8, ks, vs, bt, sl = pool(torch, cuda, 1, 128, 16, 16, [32, 16], 2, 26)
    bt[1, 1] = bt[1, 0]
    bt[0, 1] = bt[0, 0]
    q = torch.randn(2, 2, 128, generator=torch.Generator().manual_seed(8)).to(cuda)
    want = loki.dense_decode_attention_paged_q8(q, K8, V8, ks, vs, bt, torch.tensor([32, 0], dtype=torch.int32, device=cuda))
    got = loki.dense_decode_attention_paged_q8(q, K8, V8, ks, vs, bt, torch.tensor([1 << 30, -7], dtype=torch.int32, device=cuda))
    assert torch.equal(want, got) and torch.all(got[1] == 0)


def test_results_do_not_depend_on_workspace_or_stream(loki, cuda):
    """Leftovers in the workspace, another stream, a captured graph and two graphs with workspaces of
    their own: the same bits every time."""
    import torch
    K8, V8, ks, vs, bt, sl = pool(torch, cuda, 4, 128, 64, 16, [3000, 5, 0, 700], 48, 27)
    q = torch.randn(4, 16, 128, generator=torch.Generator().manual_seed(9)).to(cuda)
    idx = torch.sort(torch.randint(0, 3000, (4, 16, 300), generator=torch.Generator().manual_seed(10)), -1)[0].to(torch.int32).to(cuda)
    nd = loki.dense_decode_paged_q8_workspace_size(4, 16, 4, 64, 48, 128)
    ns = loki.loki_sparse_attention_paged_q8_workspace_size(4, 16, 4, 300, 128)

    def dense(ws=None, out=None):
        return loki.dense_decode_attention_paged_q8(q, K8, V8, ks, vs, bt, sl, workspace=ws, out=out)

    def sparse(ws=None, out=None):
        return loki.loki_sparse_attention_paged_q8(q, K8, V8, ks, vs, bt, sl, idx, dtype=torch.float32, workspace=ws, out=out)

    for f, n in ((dense, nd), (sparse, ns)):
        want = f().clone()
        for fill in (0, 255, 127):
            ws = torch.full((n,), fill, dtype=torch.uint8, device=cuda)
            assert torch.equal(f(ws), want) and torch.equal(f(ws), want)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            assert torch.equal(f(), want)
        torch.cuda.synchronize()
        graphs = []
        for _ in range(2):
            ws, out = torch.full((n,), 200, dtype=torch.uint8, device=cuda), torch.zeros_like(want)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                f(ws, out)
            graphs.append((g, ws, out))
        for s, (g, _, _) in zip((side, torch.cuda.Stream()), graphs):
            with torch.cuda.stream(s):
                for _ in range(5):
                    g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for _, _, o in graphs)


def test_pool_offsets_past_32_bits(loki, cuda):
    """Pages whose codes lie beyond 4 GiB from the pool's start."""
    import torch
    H, page, n_pages, block = 8, 256, 18000, 64  # 18000 * 8 * 256 rows of 128 bytes = 4.7 GB
    K8 = torch.zeros(n_pages, H, page, 128, dtype=torch.uint8, device=cuda).view(torch.float8_e4m3fn)
    V8 = torch.zeros_like(K8.view(torch.uint8)).view(torch.float8_e4m3fn)
    ks = torch.full((n_pages, H, page // block), 2.0 ** -7, device=cuda)
    vs = ks.clone()
    g = torch.Generator(device="cuda").manual_seed(11)
    use = [n_pages - 1, 3, n_pages - 2]
    for p in use:
        for t in (K8, V8):
            t[p] = (torch.randn(H, page, 128, generator=g, device="cuda") * 60).to(torch.float8_e4m3fn)
    bt = torch.tensor([use], dtype=torch.int32, device=cuda)
    pos, T = 700, 30
    Kn, Vn = (torch.randn(1, H, T, 128, generator=g, device="cuda") for _ in range(2))
    loki.loki_append_keys_paged_q8(Kn, Vn, None, K8, V8, ks, vs, bt, torch.tensor([pos], dtype=torch.int32, device=cuda))
    n = pos + T
    sl = torch.tensor([n], dtype=torch.int32, device=cuda)
    q = torch.randn(1, H, 128, generator=g, device="cuda")
    dense = loki.dense_decode_attention_paged_q8(q, K8, V8, ks, vs, bt, sl)
    idx = torch.arange(n, dtype=torch.int32, device=cuda).expand(1, H, n).contiguous()
    sparse = loki.loki_sparse_attention_paged_q8(q, K8, V8, ks, vs, bt, sl, idx, dtype=torch.float32)
    sub = torch.tensor(use, device=cuda)
    small = [t.view(torch.uint8)[sub].view(torch.float8_e4m3fn) for t in (K8, V8)] + [ks[sub], vs[sub]]
    bt3 = torch.arange(3, dtype=torch.int32, device=cuda)[None].contiguous()
    K, V = rows_of(small[0], small[2], bt3, 0, n, page, block), rows_of(small[1], small[3], bt3, 0, n, page, block)
    new = np.abs(K[:, pos:] - Kn[0].double().cpu().numpy())
    assert np.all(new <= np.maximum(2.0 ** -4 * np.abs(K[:, pos:]) * 1.1, 2.0 ** -16))
    for o in (dense, sparse):
        for h in range(H):
            check(o[0, h].double().cpu().numpy(), q[0, h].double().cpu().numpy(), K[h], V[h], 128 ** -0.5, 2.0 ** -24, h)


@pytest.mark.parametrize("G,D,dtn", [(1, 128, "bf16"), (4, 128, "bf16"), (2, 96, "f32")])
def test_prompt_steps_and_decodes_together(loki, cuda, G, D, dtn):
    """A run as a server makes it: a prompt's append, decode steps that append one token and attend, by
    dense attention and by Loki; every step against fp64 attention over the cache's own values, and the
    cache against the keys it was given."""
    import torch
    B, H, page, block, d, k, d_lo = 3, 2, 32, 16, 16, 40, 16
    dt = torch.bfloat16 if dtn == "bf16" else torch.float32
    half = torch.finfo(dt).eps / 2
    g = torch.Generator(device="cpu").manual_seed(31)
    rnd = lambda *s: torch.randn(*s, generator=g).to(cuda)  # noqa: E731
    T, steps, max_pages = 90, 6, 4
    lens = [90, 33, 0]
    P = torch.linalg.qr(torch.randn(H, D, D, generator=g))[0].contiguous().to(cuda)
    n_pages = B * max_pages
    bt = torch.randperm(n_pages, generator=g).to(torch.int32).view(B, max_pages).contiguous().to(cuda)
    K8 = torch.full((n_pages, H, page, D), 0x7F, dtype=torch.uint8, device=cuda).view(torch.float8_e4m3fn)
    V8 = torch.full((n_pages, H, page, D), 0x7F, dtype=torch.uint8, device=cuda).view(torch.float8_e4m3fn)
    ks = torch.full((n_pages, H, page // block), float("nan"), device=cuda)
    vs = ks.clone()
    lo = torch.full((n_pages, H, page, d_lo), float("nan"), dtype=dt, device=cuda)
    tab = loki.loki_rope_table(page * max_pages, D, device=cuda)
    sl = torch.tensor(lens, dtype=torch.int32, device=cuda)
    zero = torch.zeros_like(sl)
    loki.loki_append_keys_paged_q8(rnd(B, H, T, D).to(dt), rnd(B, H, T, D).to(dt), P, K8, V8, ks, vs, bt, zero,
                                   rope_table=tab, Kt_lo_pages=lo, new_lens=sl)
    for step in range(steps):
        Kn, Vn, qn = rnd(B, H, 1, D).to(dt), rnd(B, H, 1, D).to(dt), rnd(B, H * G, 1, D).to(dt)
        q = loki.loki_append_keys_paged_q8(Kn, Vn, P, K8, V8, ks, vs, bt, sl, rope_table=tab, Kt_lo_pages=lo, q=qn)
        sl = sl + 1
        q = q.view(B, H * G, D)
        out, idx = loki.loki_decode_attention_paged_q8(q, K8, V8, ks, vs, lo, P, bt, sl, d, k)
        q_rot = loki.loki_project_query(q, P)
        dense = loki.dense_decode_attention_paged_q8(q_rot, K8, V8, ks, vs, bt, sl)
        again = loki.loki_sparse_attention_paged_q8(q_rot, K8, V8, ks, vs, bt, sl, idx, dtype=dt)
        torch.cuda.synchronize()
        assert loki.loki_device_error(reset=True) == 0
        assert torch.equal(out, again)
        # the selection is the paged decode's own, whatever the keys and values are stored in
        wide = torch.zeros(n_pages, H, page, D, dtype=dt, device=cuda)
        _, idx2 = loki.loki_decode_attention_paged(q, wide, wide, lo, P, bt, sl, d, k)
        assert torch.equal(idx, idx2)
        qr = q_rot.double().cpu().numpy()
        for b in range(B):
            n = int(sl[b])
            K, V = rows_of(K8, ks, bt, b, n, page, block), rows_of(V8, vs, bt, b, n, page, block)
            for h in range(H * G):
                check(dense[b, h].double().cpu().numpy(), qr[b, h], K[h // G], V[h // G], D ** -0.5, 2.0 ** -24, "dense")
                i = idx[b, h].cpu().numpy()
                i = i[i >= 0]
                assert len(i) == min(k, n)
                check(out[b, h].double().cpu().numpy(), qr[b, h], K[h // G][i], V[h // G][i], D ** -0.5, half, "loki")
