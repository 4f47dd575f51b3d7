"""The forms that sizes choose between: clusters and two kernels in the 8-bit attentions, single rows
and tiles in the rotary appends, rows that leave the tiles' arithmetic. Against the fp64 restatement
in tests/q8_ref.py (GPU only)."""
from __future__ import annotations

import numpy as np
import pytest

from tests import q8_ref
from tests.test_gpu_paged_append import check_rows, expect, f64, make, places, spans, table_for
from tests.test_gpu_q8_attention import check, pool, rows_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def loki(cuda):
    import sparse_attention_decode_loki_b200 as m
    return m


# Block tables long enough that (sequences x KV heads x capacity) leaves the clusters' range, most of
# it unused: partials of many warps, of one, of none.
WIDE = [
    # H_kv, G, D, dtype, page, block, lens, pages of the table
    (1, 1, 128, "bf16", 16, 16, [5000, 1, 0, 777], 8000),
    (2, 4, 128, "f32", 64, 32, [20000, 33], 6000),
    (1, 8, 128, "bf16", 128, 64, [40000], 4000),
    (3, 5, 96, "f32", 48, 16, [1, 300, 0, 0, 2000], 4000),
    (40, 1, 128, "bf16", 32, 16, [90, 500, 31], 500),
]


@pytest.mark.parametrize("case", WIDE, ids=lambda c: "H%d-G%d-D%d-%s-n%d" % (c[0], c[1], c[2], c[3], max(c[6])))
def test_dense_q8_over_long_tables(loki, cuda, case):
    import torch
    H, G, D, dtn, page, block, lens, max_pages = case
    dt = torch.bfloat16 if dtn == "bf16" else torch.float32
    K8, V8, ks, vs, bt, sl = pool(torch, cuda, H, D, page, block, lens, max_pages, 41)
    q = torch.randn(len(lens), H * G, D, generator=torch.Generator().manual_seed(42)).to(cuda).to(dt)
    out = loki.dense_decode_attention_paged_q8(q, K8, V8, ks, vs, bt, sl)
    # the same tokens behind a table of just their pages: another form, the same answer
    short = bt[:, : max(1, -(-max(lens) // page))].contiguous()
    near = loki.dense_decode_attention_paged_q8(q, K8, V8, ks, vs, short, sl)
    torch.cuda.synchronize()
    assert loki.loki_device_error(reset=True) == 0
    o, o2, qn = (t.double().cpu().numpy() for t in (out, near, q))
    for b, n in enumerate(lens):
        K, V = rows_of(K8, ks, bt, b, n, page, block), rows_of(V8, vs, bt, b, n, page, block)
        for h in range(H * G):
            for x in (o, o2):
                check(x[b, h], qn[b, h], K[h // G], V[h // G], D ** -0.5, torch.finfo(dt).eps / 2, (b, h))


@pytest.mark.parametrize("H,G,D,lens,k", [(1, 1, 128, [3000], 400000), (2, 2, 96, [500, 0, 70], 40000), (8, 1, 128, [900] * 3, 20000)])
def test_sparse_q8_over_long_lists(loki, cuda, H, G, D, lens, k):
    """Lists with few tokens among many skipped entries, in runs and scattered, and an empty row."""
    import torch
    page, block = 64, 16
    K8, V8, ks, vs, bt, sl = pool(torch, cuda, H, D, page, block, lens, -(-max(lens) // page) + 1, 43)
    q = torch.randn(len(lens), H * G, D, generator=torch.Generator().manual_seed(44)).to(cuda)
    rng = np.random.default_rng(45)
    idx = np.full((len(lens), H * G, k), -1, np.int32)
    for b, n in enumerate(lens):
        for h in range(H * G):
            if n and not (b == 0 and h == H * G - 1 and H * G > 1):
                idx[b, h, rng.integers(0, k, 300)] = rng.integers(-1, n + 1, 300)
                idx[b, h, k // 2:k // 2 + 100] = rng.integers(0, n, 100)
    out = loki.loki_sparse_attention_paged_q8(q, K8, V8, ks, vs, bt, sl, torch.from_numpy(idx).to(cuda), dtype=torch.float32)
    torch.cuda.synchronize()
    assert loki.loki_device_error(reset=True) == 0
    o, qn = out.double().cpu().numpy(), q.double().cpu().numpy()
    for b, n in enumerate(lens):
        K, V = rows_of(K8, ks, bt, b, n, page, block), rows_of(V8, vs, bt, b, n, page, block)
        for h in range(H * G):
            i = idx[b, h]
            i = i[(i >= 0) & (i < n)]
            check(o[b, h], qn[b, h], K[h // G][i], V[h // G][i], D ** -0.5, 2.0 ** -24, (b, h))


def test_two_kernel_forms_keep_their_bits(loki, cuda):
    """Leftovers in the workspace, another stream and captured graphs side by side, each with its own
    workspace: the same bits every time."""
    import torch
    H, G, page, lens = 2, 4, 16, [7000, 12, 0]
    K8, V8, ks, vs, bt, sl = pool(torch, cuda, H, 128, page, 16, lens, 9000, 46)
    q = torch.randn(3, H * G, 128, generator=torch.Generator().manual_seed(47)).to(cuda)
    k = 30000
    idx = torch.full((3, H * G, k), -1, dtype=torch.int32, device=cuda)
    idx[0, :, ::7] = torch.randint(0, 7000, (H * G, len(range(0, k, 7))), device=cuda, dtype=torch.int32)
    nd = loki.dense_decode_paged_q8_workspace_size(3, H * G, H, page, 9000, 128)
    ns = loki.loki_sparse_attention_paged_q8_workspace_size(3, H * G, H, k, 128)
    dense = lambda ws=None, out=None: loki.dense_decode_attention_paged_q8(q, K8, V8, ks, vs, bt, sl, workspace=ws, out=out)  # noqa: E731
    sparse = lambda ws=None, out=None: loki.loki_sparse_attention_paged_q8(  # noqa: E731
        q, K8, V8, ks, vs, bt, sl, idx, dtype=torch.float32, workspace=ws, out=out)
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


def test_values_of_zero_scale_and_far_apart_scores(loki, cuda):
    """Blocks of scale zero first, then ordinary ones; scores that rise by hundreds from tile to tile."""
    import torch
    n, page = 320, 16
    K8, V8, ks, vs, bt, sl = pool(torch, cuda, 1, 128, page, 16, [n], 20, 48)
    p = bt[0, :20].long()
    vs[p[:5], :, 0] = 0.0
    q = torch.randn(1, 2, 128, generator=torch.Generator().manual_seed(49)).to(cuda)
    ks[p, 0, 0] = torch.exp2(torch.arange(20, device=cuda).float() - 8)  # scores grow to thousands
    for b2 in (bt, bt.flip(1).contiguous()):
        out = loki.dense_decode_attention_paged_q8(q, K8, V8, ks, vs, b2, sl)
        K, V = rows_of(K8, ks, b2, 0, n, page, 16), rows_of(V8, vs, b2, 0, n, page, 16)
        for h in range(2):
            check(out[0, h].double().cpu().numpy(), q[0, h].double().cpu().numpy(), K[0], V[0], 128 ** -0.5, 2.0 ** -24, h)


# --- appends ----------------------------------------------------------------------

APPENDS = [
    # B, H_kv, G, T, D, page, pos, new, dtype, basis, rot, interleaved, d_lo, block
    (1, 2, 1, 17, 128, 16, [15], [17], "bf16", True, 128, False, 128, 16),
    (1, 2, 2, 40, 128, 128, [127], [40], "f32", True, 128, True, 128, 128),
    (2, 3, 1, 260, 96, 96, [100, 0], [260, 1], "f32", True, 96, False, 96, 32),
    (30, 3, 1, 20, 128, 32, [7 * b for b in range(30)], [b % 21 for b in range(30)], "bf16", True, 64, False, 16, 32),
    (30, 3, 2, 20, 128, 32, [7 * b for b in range(30)], [b % 21 for b in range(30)], "f32", False, 64, True, 16, 16),
    (3, 40, 1, 140, 128, 64, [0, 63, 500], [140, 130, 0], "bf16", True, 0, False, 0, 64),
    (1, 3, 5, 640, 96, 64, [33], [640], "bf16", False, 96, False, 40, 64),
    (2, 2, 1, 16, 128, 16, [0, 9], [16, 11], "f32", True, 128, False, 32, 16),
    (1, 1, 1, 129, 128, 16, [127], [129], "bf16", True, 16, False, 8, 16),
]


def ids(c):
    return "B%d-H%d-T%d-D%d-p%d-%s-%s-r%d%s-lo%d-blk%d" % (c[0], c[1], c[3], c[4], c[5], c[8], "P" if c[9] else "noP",
                                                         c[10], "i" if c[11] else "", c[12], c[13])


@pytest.mark.parametrize("case", APPENDS, ids=ids)
@pytest.mark.parametrize("q8", [False, True], ids=["dt", "q8"])
def test_appends_of_all_forms(loki, cuda, case, q8):
    import torch
    B, H, G, T, D, page, pos, new, dtn, basis, rot, inter, d_lo, block = case
    dt = torch.bfloat16 if dtn == "bf16" else torch.float32
    s = make(torch, cuda, B, H, G, T, D, page, pos, new, dt, basis, rot, d_lo, block if q8 else 0, 51)
    tab = table_for(loki, cuda, max(pos) + T, rot)
    before = {k: f64(s[k]) for k in ("Kp", "Vp", "ks", "vs", "lo") if s.get(k) is not None}
    kw = dict(rope_table=tab, interleaved=inter, Kt_lo_pages=s["lo"], new_lens=s["new"], q=s["q"], q_out=torch.full_like(s["q"], 7.0))
    if q8:
        qo = loki.loki_append_keys_paged_q8(s["K"], s["V"], s["P"], s["Kp"], s["Vp"], s["ks"], s["vs"], s["bt"], s["pos"], **kw)
    else:
        qo = loki.loki_append_keys_paged_rope(s["K"], s["V"], s["P"], s["Kp"], s["Vp"], s["bt"], s["pos"], **kw)
    torch.cuda.synchronize()
    assert loki.loki_device_error(reset=True) == 0
    Kr, qr, bound = expect(s, f64(tab), inter)
    Vn, lo, qg = f64(s["V"]), f64(s["lo"]), f64(qo)
    touched = np.zeros(before["Kp"].shape[:3], bool)
    for b, t, p, slot in places(s, page):
        touched[p, :, slot] = True
        if lo is not None:
            check_rows(torch, lo[p, :, slot], Kr[b, :, t, :d_lo], dt, bound[b, :, t, :d_lo])
        if not q8:
            check_rows(torch, s["Kp"][p, :, slot].double().cpu().numpy(), Kr[b, :, t], dt, bound[b, :, t])
            assert np.array_equal(s["Vp"][p, :, slot].double().cpu().numpy(), Vn[b, :, t])
    if lo is not None:
        assert np.array_equal(lo[~touched], before["lo"][~touched])
    if not q8:
        for k in ("Kp", "Vp"):
            assert np.array_equal(f64(s[k])[~touched], before[k][~touched])
    else:
        got = {k: f64(s[k]) for k in ("Kp", "Vp", "ks", "vs")}
        want = {k: before[k].copy() for k in got}
        tol = {k: np.zeros_like(want[k]) for k in ("Kp", "Vp")}
        bt = s["bt"].cpu().numpy()
        for b in range(B):
            for h in range(H):
                for a, z in spans(pos[b], new[b], block):
                    p, at = bt[b, a // page], a % page // block
                    sl, first = slice(at * block, (at + 1) * block), a % block
                    for nm, sc, rows, bd in (("Kp", "ks", Kr, bound), ("Vp", "vs", Vn, None)):
                        x = rows[b, h, a - pos[b]:z - pos[b]]
                        codes, scale = q8_ref.append_block(want[nm][p, h, sl], want[sc][p, h, at], x, first)
                        if bd is not None:  # a key's amax must not hang on its last bits
                            top = np.abs(x).max()
                            assert abs(top / (448 * q8_ref.pow2_scale(top)) - 1) > 1e-5
                            assert abs(top / (224 * q8_ref.pow2_scale(top)) - 1) > 1e-5
                        want[nm][p, h, sl], want[sc][p, h, at] = codes, scale
                        if bd is not None:  # fp32 arithmetic may land on the code next to the exact value's
                            y, bb = x / scale, bd[b, h, a - pos[b]:z - pos[b]] / scale
                            w = codes[first:first + len(x)]
                            tol[nm][p, h, sl][first:first + len(x)] = np.maximum(
                                np.abs(q8_ref.e4m3_round(y - bb) - w), np.abs(q8_ref.e4m3_round(y + bb) - w))
        for k in ("ks", "vs"):
            assert np.array_equal(got[k], want[k]), k
        for k in ("Kp", "Vp"):
            assert np.all(np.abs(got[k] - want[k]) <= tol[k]), k
    for b in range(B):
        check_rows(torch, qg[b, :, : new[b]], qr[b, :, : new[b]], dt,
                   8 * 2.0 ** -24 * np.abs(f64(s["q"])[b, :, : new[b]]).max(-1, keepdims=True, initial=0))
        assert np.all(qg[b, :, new[b]:] == 7.0)


@pytest.mark.parametrize("T", [5, 60])
def test_infinities_and_nan_stay_in_their_rows(loki, cuda, T):
    """An infinite entry times the basis gives infinities of the basis's signs, a NaN a row of NaN; the
    other rows keep the bits they have without them. (No angles: the infinity stays in one column.)"""
    import torch
    for dt in (torch.float32, torch.bfloat16):
        def fresh(block):
            return make(torch, cuda, 1, 2, 1, T, 128, 64, [3], [T], dt, True, 0, 32, block, 53)

        def run(s):
            a = (s["K"], s["V"], s["P"], s["Kp"], s["Vp"])
            if "ks" in s:
                loki.loki_append_keys_paged_q8(*a, s["ks"], s["vs"], s["bt"], s["pos"], Kt_lo_pages=s["lo"])
            else:
                loki.loki_append_keys_paged_rope(*a, s["bt"], s["pos"], Kt_lo_pages=s["lo"])
            torch.cuda.synchronize()
            pg, slot = s["bt"][0, (3 + torch.arange(T, device=cuda)) // 64].long(), (3 + torch.arange(T, device=cuda)) % 64
            return s["Kp"][pg, :, slot].float(), s["lo"][pg, :, slot].float()

        clean, clean_lo = run(fresh(0))
        s = fresh(0)
        s["K"][0, 0, 1, 9], s["K"][0, 1, 4, 100], s["K"][0, 1, 2, 64] = float("inf"), float("-inf"), float("nan")
        K, lo = run(s)
        sign = torch.sign(s["P"])
        assert torch.equal(K[1, 0], sign[0, 9] * float("inf")) and torch.equal(K[4, 1], sign[1, 100] * float("-inf"))
        assert torch.isnan(K[2, 1]).all() and torch.isnan(lo[2, 1]).all() and torch.equal(lo[1, 0], K[1, 0, :32])
        keep = torch.ones(T, 2, dtype=torch.bool, device=cuda)
        keep[1, 0] = keep[4, 1] = keep[2, 1] = False
        assert torch.equal(K[keep], clean[keep]) and torch.equal(lo[keep], clean_lo[keep])
        s = fresh(16)
        s["K"][0, 0, 1, 9], s["K"][0, 1, 2, 64] = float("inf"), float("nan")
        codes, _ = run(s)
        assert torch.equal(codes[1, 0], sign[0, 9] * 448) and torch.isnan(codes[2, 1]).all()
        assert torch.isfinite(s["ks"]).all() and int(torch.isnan(codes).sum()) == 128


@pytest.mark.parametrize("T", [16, 50])
def test_rows_and_basis_columns_of_far_apart_sizes(loki, cuda, T):
    """Rows from 2^-60 to 2^60 and basis columns from 2^-20 to 2^20: every row and column as exact as alone."""
    import torch
    s = make(torch, cuda, 1, 2, 1, T, 128, 16, [0], [T], torch.float32, True, 128, 0, 0, 54)
    g = torch.Generator().manual_seed(55)
    s["K"] *= torch.exp2(torch.randint(-60, 61, (1, 2, T, 1), generator=g).float()).to(cuda)
    s["P"] *= torch.exp2(torch.randint(-20, 21, (2, 1, 128), generator=g).float()).to(cuda)
    tab = table_for(loki, cuda, T, 128)
    loki.loki_append_keys_paged_rope(s["K"], s["V"], s["P"], s["Kp"], s["Vp"], s["bt"], s["pos"], rope_table=tab)
    torch.cuda.synchronize()
    Kr, _, bound = expect(s, f64(tab), False)
    K = f64(s["Kp"])
    for b, t, p, slot in places(s, 16):
        check_rows(torch, K[p, :, slot], Kr[b, :, t], torch.float32, bound[b, :, t])


def test_long_append_then_attention_without_a_pause(loki, cuda):
    """A long append's two kernels, an attention that reads what they wrote, twenty times on one stream
    and in a graph: every attention sees all of its append."""
    import torch
    B, H, T, page, block = 2, 8, 700, 64, 32
    s = make(torch, cuda, B, H, 2, T, 128, page, [0, 0], [T, T - 9], torch.bfloat16, True, 128, 0, block, 56)
    tab = table_for(loki, cuda, T, 128)
    sl = s["new"].clone()
    q = torch.randn(B, 2 * H, 128, generator=torch.Generator().manual_seed(57)).to(cuda)
    names = ("Kp", "Vp", "ks", "vs")

    def step(scale, out):
        loki.loki_append_keys_paged_q8(s["K"] * scale, s["V"] * scale, s["P"], s["Kp"], s["Vp"], s["ks"], s["vs"], s["bt"],
                                       s["pos"], rope_table=tab, new_lens=s["new"])
        loki.dense_decode_attention_paged_q8(q, s["Kp"], s["Vp"], s["ks"], s["vs"], s["bt"], sl, out=out)

    outs = [torch.empty_like(q) for _ in range(20)]
    for i, o in enumerate(outs):
        step(float(i % 4 + 1), o)
    torch.cuda.synchronize()
    alone = []
    for i in range(4):
        for k in names:
            s[k].view(torch.uint8).fill_(0x11) if k in ("Kp", "Vp") else s[k].fill_(1.0)
        torch.cuda.synchronize()
        o = torch.empty_like(q)
        step(float(i + 1), o)
        torch.cuda.synchronize()
        alone.append(o)
    assert all(torch.equal(o, alone[i % 4]) for i, o in enumerate(outs))
    g, o = torch.cuda.CUDAGraph(), torch.empty_like(q)
    with torch.cuda.graph(g):
        step(3.0, o)
    for _ in range(3):
        o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, alone[2])
    assert loki.loki_device_error(reset=True) == 0


def test_calls_behind_copies_other_streams_and_joins(loki, cuda):
    """The kernels are launched before their predecessors end and wait for them: inputs made just before
    the call by a kernel, a copy, a fill or another stream, eager and captured with two streams joined."""
    import torch
    B, H, page, n = 3, 4, 32, 500
    K8, V8, ks, vs, bt, sl = pool(torch, cuda, H, 128, page, 16, [n, 40, 0], 16, 58)
    src = torch.randn(6, B, 2 * H, 128, generator=torch.Generator().manual_seed(59)).to(cuda)
    host = src.cpu().pin_memory()
    want = [loki.dense_decode_attention_paged_q8(x.contiguous(), K8, V8, ks, vs, bt, sl).clone() for x in src]
    zero = loki.dense_decode_attention_paged_q8(torch.zeros_like(src[0]), K8, V8, ks, vs, bt, sl).clone()
    torch.cuda.synchronize()
    q, out = torch.empty_like(src[0]), torch.empty_like(src[0])
    big = torch.zeros(64 << 20, device=cuda)
    side = torch.cuda.Stream()

    def call():
        return loki.dense_decode_attention_paged_q8(q, K8, V8, ks, vs, bt, sl, out=out)

    got = []
    for i in range(6):
        big.add_(1.0)  # keeps the device busy, so that what follows is queued
        q.copy_(src[i])
        got.append(call().clone())
        big.add_(1.0)
        q.copy_(host[i], non_blocking=True)
        got.append(call().clone())
        big.add_(1.0)
        q.zero_()
        got.append(call().clone())
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            big.add_(1.0)
            q.copy_(src[(i + 1) % 6])
        torch.cuda.current_stream().wait_stream(side)
        got.append(call().clone())
    torch.cuda.synchronize()
    for i in range(6):
        for g, w in zip(got[4 * i:4 * i + 4], (want[i], want[i], zero, want[(i + 1) % 6])):
            assert torch.equal(g, w), i

    T = 40
    s = make(torch, cuda, 1, 2, 2, T, 128, 16, [0], [T], torch.bfloat16, True, 128, 32, 16, 60)
    one = make(torch, cuda, 1, 2, 2, 1, 128, 16, [T], [1], torch.bfloat16, True, 128, 32, 0, 61)
    bt2 = torch.arange(3, dtype=torch.int32, device=cuda)[None].contiguous()
    tab = table_for(loki, cuda, T + 1, 128)
    pages = [torch.zeros(3, 2, 16, 128, dtype=torch.uint8, device=cuda).view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.ones(3, 2, 1, device=cuda) for _ in range(2)]
    length = torch.zeros(1, dtype=torch.int32, device=cuda)
    qo, ao = torch.empty_like(one["q"]), torch.empty(1, 4, 128, device=cuda, dtype=torch.bfloat16)

    def steps():
        length.zero_()
        loki.loki_append_keys_paged_q8(s["K"], s["V"], s["P"], *pages, *scales, bt2, length, rope_table=tab)
        length.add_(T)
        loki.loki_append_keys_paged_q8(one["K"], one["V"], s["P"], *pages, *scales, bt2, length, rope_table=tab, q=one["q"], q_out=qo)
        length.add_(1)
        loki.dense_decode_attention_paged_q8(qo.view(1, 4, 128), *pages, *scales, bt2, length, out=ao)

    def result():
        torch.cuda.synchronize()
        return [t.view(torch.uint8).clone() if t.dtype == torch.float8_e4m3fn else t.clone() for t in (*pages, *scales, qo, ao)]

    steps()
    eager = result()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            big[:1024].add_(1.0)
        big[2048:4096].add_(1.0)
        torch.cuda.current_stream().wait_stream(side)  # two nodes before the first call
        steps()
        steps()
    for _ in range(3):
        for t in (*pages, *scales, qo, ao):
            (t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t).zero_()
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(result(), eager))
    assert loki.loki_device_error(reset=True) == 0


def test_tensors_without_memory_are_an_error(loki, cuda):
    """Tensors that stand for shapes only (their addresses cannot be read): an exception, no launch."""
    import torch
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        q = torch.empty(1, 2, 128, device=cuda)
        p8 = torch.empty(2, 2, 16, 128, device=cuda, dtype=torch.float8_e4m3fn)
        sc = torch.empty(2, 2, 1, device=cuda)
        bt, n = (torch.empty(*s, device=cuda, dtype=torch.int32) for s in ((1, 2), (1,)))
        idx = torch.empty(1, 2, 4, device=cuda, dtype=torch.int32)
        plane, P = torch.empty(2, 2, 16, 16, device=cuda), torch.empty(2, 128, 128, device=cuda)
        new, tab = torch.empty(1, 2, 1, 128, device=cuda), torch.empty(8, 128, device=cuda)
    pages = (p8, p8, sc, sc, bt, n)
    for call in (lambda: loki.dense_decode_attention_paged_q8(q, *pages),
                 lambda: loki.loki_sparse_attention_paged_q8(q, *pages, idx),
                 lambda: loki.loki_decode_attention_paged_q8(q, *pages[:4], plane, P, bt, n, 16, 4),
                 lambda: loki.loki_append_keys_paged_q8(new, new, P, *pages, rope_table=tab),
                 lambda: loki.loki_append_keys_paged_rope(new, new, P, plane.new_empty(2, 2, 16, 128),
                                                          plane.new_empty(2, 2, 16, 128), bt, n)):
        with pytest.raises((RuntimeError, ValueError)):  # (a null address, or one that the type refuses to give)
            call()
    torch.cuda.synchronize()
    assert loki.loki_device_error(reset=True) == 0


@pytest.mark.parametrize("T", [16, 17, 300])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("q8", [False, True], ids=["dt", "q8"])
def test_queries_in_place_in_all_forms(loki, cuda, T, inter, q8):
    """q_out may be q: the same bits, in single rows, tiles and streams, tokens left out included."""
    import torch
    lens = [T, 0, T // 2]
    s = make(torch, cuda, 3, 2, 4, T, 128, 64, [0, 5, 40], lens, torch.bfloat16, q8, 96, 0, 16 if q8 else 0, 51)
    tab = table_for(loki, cuda, 512, 96)
    for P in (None, s["P"]):
        pages = (s["Kp"], s["Vp"]) + ((s["ks"], s["vs"]) if q8 else ())
        f = loki.loki_append_keys_paged_q8 if q8 else loki.loki_append_keys_paged_rope
        q = s["q"].clone()
        apart = q.clone()
        kw = dict(rope_table=tab, interleaved=inter, new_lens=s["new"])
        f(s["K"], s["V"], P, *pages, s["bt"], s["pos"], q=s["q"], q_out=apart, **kw)
        got = f(s["K"], s["V"], P, *pages, s["bt"], s["pos"], q=q, q_out=q, **kw)
        assert got is q and torch.equal(q, apart) and torch.equal(q[1], s["q"][1])


@pytest.mark.parametrize("what", ["rope_table", "Kt_lo_pages", "new_lens", "q"])
def test_empty_optional_tensors_are_refused(loki, cuda, what):
    """An empty table is no missing table: nothing is appended unrotated."""
    import torch
    s = make(torch, cuda, 1, 2, 1, 3, 128, 16, [0], [3], torch.bfloat16, False, 128, 0, 0, 61)
    was = s["Kp"].clone()
    empty = {"rope_table": torch.empty(0, 128, device=cuda), "Kt_lo_pages": s["Kp"][..., :0].contiguous(),
             "new_lens": s["new"][:0], "q": s["q"][:, :0]}[what]
    with pytest.raises(ValueError):
        loki.loki_append_keys_paged_rope(s["K"], s["V"], None, s["Kp"], s["Vp"], s["bt"], s["pos"], **{what: empty})
    assert torch.equal(s["Kp"], was)


@pytest.mark.parametrize("T", [12, 40])
@pytest.mark.parametrize("D,dtn", [(128, "bf16"), (96, "bf16"), (128, "f32")])
def test_queries_at_the_ends_of_the_positions(loki, cuda, T, D, dtn):
    """Positions below zero or behind the angle table, and new_lens, cut a sequence's rows anywhere: the
    others' queries are turned, theirs are left."""
    import torch
    dt = torch.bfloat16 if dtn == "bf16" else torch.float32
    pos, new, n_pos = [-3, 7, -50, 0, -6], [T, T - 5, T, 3, T], 7 + T - 9
    s = make(torch, cuda, 5, 2, 3, T, D, 16, [0] * 5, [0] * 5, dt, False, 96, 0, 0, 71)
    s["bt"].fill_(-1)  # no pages: only the queries have a place to go
    tab = table_for(loki, cuda, n_pos, 96)
    q_out = torch.full_like(s["q"], 7.0)
    i32 = lambda x: torch.tensor(x, device=cuda, dtype=torch.int32)  # noqa: E731
    loki.loki_append_keys_paged_rope(s["K"], s["V"], None, s["Kp"], s["Vp"], s["bt"], i32(pos), rope_table=tab,
                                     new_lens=i32(new), q=s["q"], q_out=q_out)
    torch.cuda.synchronize()
    loki.loki_device_error(reset=True)  # (tokens without a place are flagged)
    q, got, t64 = f64(s["q"]), f64(q_out), f64(tab)
    for b in range(5):
        for t in range(T):
            j = pos[b] + t
            if j < 0 or j >= n_pos or t >= new[b]:
                assert np.all(got[b, :, t] == 7.0), (b, t)
                continue
            x, c, sn = q[b, :, t], t64[j, :48], t64[j, 48:]
            want = x.copy()
            want[:, :48] = x[:, :48] * c - x[:, 48:96] * sn
            want[:, 48:96] = x[:, :48] * sn + x[:, 48:96] * c
            # two fp32 roundings of products of two, then one to dt
            check_rows(torch, got[b, :, t], want, dt, 2.0 ** -23 * 2 * np.abs(x).max())


@pytest.mark.parametrize("dtn,H,T", [("f32", 40, 2312), ("bf16", 32, 4096)])
def test_queries_of_long_prompts_call_after_call(loki, cuda, dtn, H, T):
    """Many heads of rows that stay in the cache, again and again: the rings' slots are read before they
    are filled anew."""
    import torch
    dt = torch.bfloat16 if dtn == "bf16" else torch.float32
    s = make(torch, cuda, 1, 8, H // 8, T, 128, 48, [20], [T], dt, False, 128, 32, 0, 81)
    tab = table_for(loki, cuda, 20 + T, 128)
    outs = torch.zeros(60, *s["q"].shape, device=cuda, dtype=dt) if dtn == "bf16" else torch.zeros(40, *s["q"].shape, device=cuda)
    for o in outs:
        loki.loki_append_keys_paged_rope(s["K"], s["V"], None, s["Kp"], s["Vp"], s["bt"], s["pos"], rope_table=tab,
                                         Kt_lo_pages=s["lo"], q=s["q"], q_out=o)
    x, c, sn = s["q"].double(), tab[20:, :64].double(), tab[20:, 64:].double()
    want = torch.cat([x[..., :64] * c - x[..., 64:] * sn, x[..., :64] * sn + x[..., 64:] * c], dim=-1)
    # fp32: two roundings of at most |a c| + |b s| each; then one to dt
    bound = 2.0 ** -23 * 2 * float(x.abs().max())
    tol = torch.finfo(dt).eps / 2 * (want.abs() + bound) + bound
    for i, o in enumerate(outs):
        assert bool(((o.double() - want).abs() <= tol).all()), i


def test_first_calls_of_new_processes(cuda):
    """The first call of a process, its memory and code cold, is where a slot filled too early showed."""
    import os
    import subprocess
    import sys
    code = """
import torch, sparse_attention_decode_loki_b200 as loki
g = torch.Generator().manual_seed(91)
T, H = 2312, 40
q = torch.randn(1, H, T, 128, generator=g).cuda()
new = torch.randn(1, 8, T, 128, generator=g).cuda()
pages = torch.zeros(49, 8, 48, 128, device="cuda")
tab = loki.loki_rope_table(T, 128, device="cuda")
bt, pos = torch.arange(49, device="cuda", dtype=torch.int32)[None], torch.zeros(1, device="cuda", dtype=torch.int32)
got = loki.loki_append_keys_paged_rope(new, new, None, pages, pages.clone(), bt, pos, rope_table=tab, q=q)
x, c, s = q.double(), tab[:, :64].double(), tab[:, 64:].double()
want = torch.cat([x[..., :64] * c - x[..., 64:] * s, x[..., :64] * s + x[..., 64:] * c], dim=-1)
bound = 2.0 ** -22 * float(x.abs().max())  # three fp32 roundings of at most |a c| + |b s| each
assert bool(((got.double() - want).abs() <= bound).all())
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    for _ in range(2):
        jobs = [subprocess.Popen([sys.executable, "-c", code], cwd=root) for _ in range(4)]
        assert [j.wait(timeout=300) for j in jobs] == [0] * 4
