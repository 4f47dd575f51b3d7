"""Refusals of the rotary paged appends and the 8-bit attentions, and the fp64 restatement's own
pins. No GPU: pointers are fake and every call fails its checks before any CUDA call."""
import numpy as np
import pytest

from tests import q8_ref

F = 1 << 20


@pytest.fixture(scope="module")
def L():
    from sparse_attention_decode_loki_b200 import _lib
    return _lib


def append(L, q8, **kw):
    a = dict(K=F, V=F, P=F, rope=F, n_pos=64, rot=128, inter=0, q=F, q_out=F, H_q=4, Kp=F, Vp=F, ks=F,
             vs=F, block=16, lo=F, d_lo=32, bt=F, pos=F, new=F, B=2, H_kv=2, T=3, page=16, max_pages=4,
             n_pages=8, D=128, dt=L.DTYPE_BF16)
    a.update(kw)
    front = [a[k] for k in ("K", "V", "P", "rope", "n_pos", "rot", "inter", "q", "q_out", "H_q", "Kp", "Vp")]
    back = [a[k] for k in ("lo", "d_lo", "bt", "pos", "new", "B", "H_kv", "T", "page", "max_pages",
                           "n_pages", "D", "dt")]
    if q8:
        return L.lib.loki_append_keys_paged_q8(*front, a["ks"], a["vs"], a["block"], *back, None)
    return L.lib.loki_append_keys_paged_rope(*front, *back, None)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(K=None), 1), (dict(V=F + 8), 1), (dict(P=F + 4), 1), (dict(rope=F + 4), 1), (dict(n_pos=0), 1),
    (dict(rot=24), 1), (dict(rot=0), 1), (dict(rot=144), 1), (dict(rot=112, D=96), 1), (dict(q=None), 1),
    (dict(q_out=None), 1), (dict(q=F + 2), 1), (dict(H_q=3), 1), (dict(H_q=18), 2), (dict(Kp=None), 1),
    (dict(Vp=F + 1), 1), (dict(lo=F + 8), 1), (dict(d_lo=12), 1), (dict(d_lo=136), 1), (dict(bt=None), 1),
    (dict(pos=F + 2), 1), (dict(new=F + 1), 1), (dict(B=0), 1), (dict(H_kv=0), 1), (dict(T=0), 1),
    (dict(page=0), 1), (dict(max_pages=0), 1), (dict(n_pages=0), 1), (dict(n_pages=1 << 40), 2),
    (dict(D=64), 2), (dict(dt=5), 1), (dict(page=1 << 20, max_pages=1 << 12), 2),
])
def test_appends_refuse(L, q8, kw, status):
    assert append(L, q8, **kw) == status
    assert L.lib.loki_last_error().decode() != ""


@pytest.mark.parametrize("kw", [dict(block=0), dict(block=8), dict(block=48, page=48), dict(block=32), dict(ks=None),
                                dict(vs=F + 2), dict(block=256, page=256)])
def test_q8_append_refuses_blocks_and_scales(L, kw):
    assert append(L, True, **kw) == 1


def attend(L, kind, **kw):
    a = dict(q=F, K=F, V=F, ks=F, vs=F, block=16, lo=F, d_lo=32, P=F, bt=F, sl=F, idx=F, B=2, H_q=4, H_kv=2,
             page=16, max_pages=4, n_pages=8, D=128, d=32, k=20, dt=L.DTYPE_BF16, out=F, ws=F, ws_bytes=None)
    a.update(kw)
    lib = L.lib
    head = [a[k] for k in ("q", "K", "V", "ks", "vs", "block")]
    size = [a[k] for k in ("B", "H_q", "H_kv", "page", "max_pages", "n_pages", "D")]
    if kind == "dense":
        need = lib.dense_decode_paged_q8_workspace_size(a["B"], a["H_q"], a["H_kv"], a["page"], a["max_pages"], a["D"])
        wb = need + (a["ws_bytes"] or 0)
        return lib.dense_decode_attention_paged_q8(*head, a["bt"], a["sl"], *size, 0.0, a["dt"], a["out"], a["ws"], wb, None)
    if kind == "sparse":
        need = lib.loki_sparse_attention_paged_q8_workspace_size(a["B"], a["H_q"], a["H_kv"], a["k"], a["D"])
        wb = need + (a["ws_bytes"] or 0)
        return lib.loki_sparse_attention_paged_q8(*head, a["bt"], a["sl"], a["idx"], *size, a["k"], 0.0, a["dt"], a["out"], a["ws"], wb, None)
    need = lib.loki_paged_q8_decode_workspace_size(a["B"], a["H_q"], a["H_kv"], a["page"], a["max_pages"], a["D"], a["d"], a["k"])
    wb = need + (a["ws_bytes"] or 0)
    return lib.loki_decode_attention_paged_q8(*head, a["lo"], a["d_lo"], a["P"], a["bt"], a["sl"], *size, a["d"], a["k"], 0.0,
                                              a["dt"], a["out"], a["idx"], a["ws"], wb, None)


@pytest.mark.parametrize("kind", ["dense", "sparse", "decode"])
@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(K=F + 8), 1), (dict(V=None), 1), (dict(ks=None), 1), (dict(vs=F + 2), 1),
    (dict(block=0), 1), (dict(block=24, page=24), 1), (dict(block=32), 1), (dict(bt=None), 1),
    (dict(sl=F + 2), 1), (dict(B=0), 1), (dict(H_q=3), 1), (dict(H_q=18), 2), (dict(D=64), 2),
    (dict(page=0), 1), (dict(n_pages=0), 1), (dict(n_pages=1 << 40), 2), (dict(dt=9), 1),
    (dict(out=F + 2), 1), (dict(out=None), 1), (dict(ws=None), 1), (dict(ws=F + 16), 1), (dict(ws_bytes=-1), 3),
])
def test_attentions_refuse(L, kind, kw, status):
    assert attend(L, kind, **kw) == status
    assert L.lib.loki_last_error().decode() != ""


@pytest.mark.parametrize("kind,kw,status", [
    ("sparse", dict(k=0), 1), ("sparse", dict(idx=None), 1), ("sparse", dict(idx=F + 2), 1), ("decode", dict(k=65), 1),
    ("decode", dict(k=0), 1), ("decode", dict(d=33), 1), ("decode", dict(d_lo=20, d=16), 1), ("decode", dict(lo=None), 1),
    ("decode", dict(P=F + 4), 1), ("decode", dict(idx=None), 1), ("decode", dict(H_q=16, H_kv=2, d_lo=32), 2),
    ("decode", dict(page=4096, max_pages=128, k=64), 2),
])
def test_selected_attentions_refuse(L, kind, kw, status):
    assert attend(L, kind, **kw) == status


@pytest.mark.parametrize("args,status", [
    ((F, 0, 128, 10000.0, 1.0), 1), ((F, 8, 24, 10000.0, 1.0), 1), ((F, 8, 144, 10000.0, 1.0), 1),
    ((F, 8, 64, 0.0, 1.0), 1), ((F, 8, 64, float("inf"), 1.0), 1), ((F, 8, 64, 10000.0, float("nan")), 1),
    ((None, 8, 64, 10000.0, 1.0), 1), ((F + 4, 8, 64, 10000.0, 1.0), 1),
])
def test_rope_table_refuses(L, args, status):
    assert L.lib.loki_rope_table(*args, None) == status


def test_workspace_sizes_of_nonsense_are_zero(L):
    assert L.lib.dense_decode_paged_q8_workspace_size(0, 1, 1, 16, 1, 128) == 0
    assert L.lib.loki_sparse_attention_paged_q8_workspace_size(1, 1, 1, 0, 128) == 0
    assert L.lib.loki_paged_q8_decode_workspace_size(1, 1, 0, 16, 1, 128, 32, 4) == 0


def test_python_wants_cuda_tensors_and_types():
    torch = pytest.importorskip("torch")
    import sparse_attention_decode_loki_b200 as loki
    q = torch.zeros(1, 1, 128)
    pg = torch.zeros(1, 1, 16, 128, dtype=torch.float8_e4m3fn)
    sc = torch.ones(1, 1, 1)
    bt, sl = torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        loki.dense_decode_attention_paged_q8(q, pg, pg, sc, sc, bt, sl)
    with pytest.raises(TypeError):
        loki.dense_decode_attention_paged_q8(q, pg.view(torch.uint8), pg, sc, sc, bt, sl)
    with pytest.raises(ValueError):
        loki.dense_decode_attention_paged_q8(q, pg, pg, torch.ones(1, 1, 3), sc, bt, sl)
    with pytest.raises(ValueError):
        loki.loki_append_keys_paged_rope(q[None], q[None], None, q[None], q[None], bt, sl)


def test_binding_refuses_what_is_no_tensor_or_number():
    torch = pytest.importorskip("torch")
    import sparse_attention_decode_loki_b200 as loki
    from sparse_attention_decode_loki_b200 import _binding as b
    t = torch.zeros(1, 1, 16, 128)
    p8 = t.to(torch.float8_e4m3fn)
    sc, bt = torch.ones(1, 1, 1), torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(TypeError):
        b.dense(t)
    with pytest.raises(TypeError, match="q must be a tensor"):
        loki.dense_decode_attention_paged_q8(3, p8, p8, sc, sc, bt, bt[0])
    with pytest.raises(TypeError, match="float8"):
        loki.loki_append_keys_paged_q8(t, t, None, t, t, sc, sc, bt, bt[0])
    with pytest.raises(TypeError, match="v_scales must be a tensor"):
        loki.loki_append_keys_paged_q8(t, t, None, p8, p8, sc, None, bt, bt[0])
    with pytest.raises(ValueError, match="v_scales must be torch.float32 \\[1, 1, 1\\]"):
        loki.loki_append_keys_paged_q8(t, t, None, p8, p8, sc, sc.double(), bt, bt[0])
    with pytest.raises(ValueError, match="CUDA tensors"):
        loki.loki_append_keys_paged_rope(t, t, None, t, t, bt, bt[0])
    with pytest.raises(ValueError, match="CUDA tensors"):
        b.rope_table(torch.zeros(4, 16), 10000.0, 1.0)


# --- the restatement's own pins -------------------------------------------------

def test_e4m3_rounding_agrees_with_the_type():
    torch = pytest.importorskip("torch")
    x = torch.cat([torch.randn(20000, generator=torch.Generator().manual_seed(1)) * 10 ** e for e in (-4, -2, 0, 2)])
    x = torch.cat([x.clamp(-448, 448), torch.tensor([0.0, -0.0, 448.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 17.0, 19.0])])
    assert np.array_equal(q8_ref.e4m3_round(x.double().numpy()), x.to(torch.float8_e4m3fn).double().numpy())


def test_scale_is_the_least_power_of_two():
    for amax in (448.0, 448.0000001, 449.0, 1.0, 1e-30, 3e38, 0.4375, 2.0 ** -140):
        s = q8_ref.pow2_scale(amax)
        assert amax <= 448 * s and (s == 2.0 ** -126 or amax > 224 * s)
    assert q8_ref.pow2_scale(0.0) == 2.0 ** -126


def test_attend_by_hand():
    K, V = np.array([[1.0, 0.0], [0.0, 1.0]]), np.array([[2.0, 0.0], [0.0, 4.0]])
    assert np.allclose(q8_ref.attend(np.array([np.log(3.0), 0.0]), K, V, 1.0), [1.5, 1.0])
    assert np.array_equal(q8_ref.attend(np.ones(2), K[:0], V[:0], 1.0), np.zeros(2))


def test_append_block_by_hand():
    codes = np.zeros((16, 1))
    codes[0] = 448.0
    new, s = q8_ref.append_block(codes, 1.0, np.array([[900.0]]), 1)
    assert s == 4.0 and new[0] == 112.0 and new[1] == 224.0  # 900 needs 448 * 4; 225 rounds to 224
    new, s = q8_ref.append_block(codes, 8.0, np.array([[900.0]]), 0)
    assert s == 4.0 and new[0] == 224.0  # first row: the old scale does not count
