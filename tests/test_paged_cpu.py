"""Paged cache and delta rule on the host: oracle pins, refusals of the C entry points and of the classes' calls.
No kernel is launched here."""

import ctypes

import numpy as np
import pytest

from oracle import delta as OD
from oracle import paged as OP


# ---- the oracle ------------------------------------------------------------------------------------
def test_e4m3_codes_round_to_nearest_even():
    vals = OP.e4m3_values()
    fin = np.where(np.isfinite(vals))[0]
    assert vals[126] == 448 and vals[1] == 2.0 ** -9 and np.isnan(vals[127]) and np.isnan(vals[255])
    assert np.array_equal(OP.encode(vals[fin], "e4m3"), fin)
    pos = vals[:127]
    mid = (pos[:-1] + pos[1:]) / 2
    assert np.array_equal(OP.encode(mid, "e4m3"), np.where(np.arange(126) % 2 == 0, np.arange(126), np.arange(1, 127)))
    rng = np.random.default_rng(0)
    y = rng.standard_normal(2000) * np.exp(rng.uniform(-8, 6, 2000))
    got = vals[OP.encode(y, "e4m3")]
    best = pos[np.abs(np.abs(y)[:, None] - pos).argmin(1)] * np.sign(y)
    assert np.array_equal(np.abs(got - y), np.abs(best - y))
    assert vals[OP.encode(np.array([1e9, -np.inf, np.nan]), "e4m3")].tolist() == [448.0, -448.0, 0.0]
    assert OP.values(OP.encode(np.array([1e9, -1e9, 0.5, 1.5, np.nan]), "int8"), "int8").tolist() == [127, -127, 0, 2, 0]


def test_e4m3_bytes_are_torchs():
    import torch
    rng = np.random.default_rng(1)
    y = np.concatenate([rng.standard_normal(4000) * 20, rng.uniform(-0.02, 0.02, 500), [0.0, -0.0, 448.0]]).astype(np.float32)
    t = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(OP.encode(y.astype(np.float64), "e4m3"), t)


def test_scale_is_the_smallest_that_holds():
    for amax in (448.0, 448.1, 224.0, 1e-3, 3.4e38):
        s = OP.scale_for(amax, "e4m3")
        assert 448 * s >= amax and 448 * s / 2 < amax
    assert OP.scale_for(0.0, "e4m3") == OP.scale_for(0.0, "int8") == 2.0 ** -126


def test_rotation_is_a_rotation():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((5, 2, 64))
    ang = rng.uniform(0, 6, (9, 16))
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    for inter in (False, True):
        y = OP.rotate(x, table, np.arange(3, 8), inter)
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
        assert np.array_equal(y[..., 32:], x[..., 32:])
        z = x[..., 0:32:2] + 1j * x[..., 1:32:2] if inter else x[..., :16] + 1j * x[..., 16:32]
        w = y[..., 0:32:2] + 1j * y[..., 1:32:2] if inter else y[..., :16] + 1j * y[..., 16:32]
        assert np.allclose(w, z * np.exp(1j * ang[3:8])[:, None])


def test_attention_special_cases():
    rng = np.random.default_rng(3)
    K, V = rng.standard_normal((7, 1, 4)), rng.standard_normal((7, 1, 4))
    q = np.zeros((2, 2, 4))
    out, lse, _, _ = OP.attend(q, K, V, 2, 7, 0.5)
    assert np.allclose(out[1], V[:, 0].mean(0)) and np.allclose(out[0], V[:6, 0].mean(0)) and np.allclose(lse[1], np.log(7))
    out, lse, _, _ = OP.attend(q, K, V, 2, 7, 0.5, window=2, n_sink=1)
    assert np.allclose(out[1], V[[0, 5, 6], 0].mean(0)) and np.allclose(lse, np.log(3))
    out, lse, _, _ = OP.attend(np.zeros((3, 1, 4)), K[:1], V[:1], 3, 1, 0.5)   # two rows before the sequence's begin
    assert np.array_equal(out[:2], np.zeros((2, 1, 4))) and np.isneginf(lse[:2]).all() and lse[2] == 0


def test_delta_rule_special_cases():
    rng = np.random.default_rng(4)
    k = rng.standard_normal((3, 1, 8))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    v, S = rng.standard_normal((3, 2, 5)), rng.standard_normal((2, 8, 5))
    one, zero = np.ones((3, 2)), np.zeros((3, 2))
    out, T, _ = OD.run(S, k, k, v, zero, one, 1.0)          # beta = 1, unit keys: reading a key gives its value
    assert np.allclose(out, v)
    out, T, _ = OD.run(S, k, k, v, zero, zero, 1.0)         # beta = 0: nothing is written
    assert np.allclose(T, S)
    _, T, _ = OD.run(S, k[:1], k[:1], v[:1], np.full((1, 2), -np.inf), one[:1], 1.0)   # all forgotten
    assert np.allclose(T, k[0, 0][None, :, None] * v[0][:, None, :])


# ---- refusals of the C entry points ------------------------------------------------------------------
@pytest.fixture(scope="module")
def A():
    from hybrid_sparse_linear_decode_b200 import build
    build.build()
    from hybrid_sparse_linear_decode_b200 import _abi
    _abi.load_library()
    return _abi


def _cache(A, **kw):
    c = dict(k_codes=256, v_codes=512, k_scales=1024, v_scales=2048, n_pages=8, n_kv_heads=2, page_size=16, head_dim=64, code=0)
    c.update(kw)
    return A.hyb_attn_paged_cache(**c)


def _batch(A, **kw):
    b = dict(page_table=64, cu_new=64, kv_lens=64, batch=2, table_stride=4, n_new=2, max_new=1, max_len=64, status=None)
    b.update(kw)
    return A.hyb_attn_paged_batch(**b)


BAD_CACHE = [dict(n_pages=1 << 26, n_kv_heads=4), dict(n_pages=(1 << 31) - 1, page_size=256), dict(head_dim=96), dict(page_size=8), dict(page_size=24), dict(page_size=272), dict(n_pages=0), dict(n_kv_heads=0),
             dict(code=2)]
BAD_BATCH = [dict(batch=0), dict(table_stride=0), dict(table_stride=1 << 27), dict(n_new=-1), dict(max_new=3), dict(max_new=0),
             dict(max_len=-1), dict(batch=40000), dict(batch=30000, table_stride=1 << 18)]
BAD_POINTERS = [dict(k_codes=None), dict(v_codes=None), dict(k_codes=8), dict(k_scales=None), dict(v_scales=2)]
BAD_ARRAYS = [dict(page_table=None), dict(cu_new=None), dict(kv_lens=None), dict(cu_new=2), dict(status=2)]


@pytest.mark.parametrize("cache,batch", [(c, {}) for c in BAD_CACHE + BAD_POINTERS] + [({}, b) for b in BAD_BATCH + BAD_ARRAYS])
def test_paged_calls_refuse_bad_descriptions(A, cache, batch):
    c, b = _cache(A, **cache), _batch(A, **batch)
    for call in (lambda: A.hyb_attn_paged_append(c, b, 0, 256, 128, 512, 128, None, 0, 0, 0, None, 0, None, 0, 0, None),
                 lambda: A.hyb_attn_paged_attend(c, b, 0, 256, 256, 512, 256, None, 4, 0, 0, 0.0, 1024, 1 << 30, None)):
        with pytest.raises(A.HybAttnError) as e:
            call()
        assert e.value.code == A.HYB_EINVAL
    if cache not in BAD_POINTERS and batch not in BAD_ARRAYS:
        assert A.hyb_attn_paged_workspace_size(c, b, 4) == 0


@pytest.mark.parametrize("kw", [dict(type=2), dict(k=None), dict(k=8), dict(v=None), dict(k_stride=120), dict(k_stride=132),
                                dict(rope=24, n_pos=4, rot_dim=32), dict(rope=256, n_pos=0, rot_dim=32),
                                dict(rope=256, n_pos=4, rot_dim=24), dict(rope=256, n_pos=4, rot_dim=80), dict(q=256),
                                dict(q_out=256), dict(q=256, q_out=256, n_q_heads=0), dict(q=256, q_out=256, q_stride=264),
                                dict(q=256, q_out=256, q_out_stride=192)])
def test_append_refuses_bad_rows(A, kw):
    a = dict(type=0, k=256, k_stride=128, v=512, v_stride=128, rope=None, n_pos=0, rot_dim=0, interleaved=0, q=None, q_stride=256,
             q_out=None, q_out_stride=256, n_q_heads=4, stream=None)
    a.update(kw)
    with pytest.raises(A.HybAttnError) as e:
        A.hyb_attn_paged_append(_cache(A), _batch(A), **a)
    assert e.value.code == A.HYB_EINVAL


@pytest.mark.parametrize("kw,code", [(dict(type=-1), -1), (dict(n_q_heads=3), -1), (dict(n_q_heads=0), -1), (dict(q=None), -1),
                                     (dict(q_stride=250), -1), (dict(q_stride=252), -1), (dict(out=None), -1), (dict(out_stride=254), -1),
                                     (dict(window=-1), -1), (dict(n_sink=-1), -1), (dict(scale=-1.0), -1),
                                     (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(lse=2), -1),
                                     (dict(workspace=None), -6), (dict(workspace_bytes=16), -6), (dict(workspace=8), -1)])
def test_attend_refuses_bad_rows(A, kw, code):
    a = dict(type=0, q=256, q_stride=256, out=512, out_stride=256, lse=None, n_q_heads=4, window=0, n_sink=0, scale=0.0,
             workspace=1024, workspace_bytes=1 << 30, stream=None)
    a.update(kw)
    with pytest.raises(A.HybAttnError) as e:   # long enough that the parts of a sequence go through the workspace
        A.hyb_attn_paged_attend(_cache(A), _batch(A, table_stride=4096, max_len=65536), **a)
    assert e.value.code == code


def test_no_new_rows_is_no_work(A):
    c, b = _cache(A), _batch(A, n_new=0, max_new=0)
    A.hyb_attn_paged_append(c, b, 0, None, 0, None, 0, None, 0, 0, 0, None, 0, None, 0, 0, None)
    A.hyb_attn_paged_attend(c, b, 0, None, 0, None, 0, None, 4, 0, 0, 0.0, None, 0, None)
    assert A.hyb_attn_paged_workspace_size(c, b, 4) == 0


@pytest.mark.parametrize("B,new,G", [(1, 1, 1), (3, 4, 4), (8, 1, 4), (100, 1, 4), (2, 40, 8), (64, 1, 8), (1, 700, 1), (2, 1500, 8), (8, 600, 4)])
def test_workspace_of_a_window_fits_the_workspace_asked_for(A, B, new, G):
    """The workspace size does not depend on the window, which only shrinks the work: a call with one takes the same
    buffer (it reaches the launch, which fails here without a GPU, instead of the workspace check)."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    for pages in (1, 7, 33, 90, 257, 600, 2000):
        c, b = _cache(A), _batch(A, batch=B, n_new=B * new, max_new=new, table_stride=pages, max_len=16 * pages)
        size = A.hyb_attn_paged_workspace_size(c, b, 2 * G)
        for window in (0, 1, 100, 1000, 5000, 1 << 30):
            with pytest.raises(A.HybAttnError) as e:
                A.hyb_attn_paged_attend(c, b, 0, 256, 128 * G, 512, 128 * G, None, 2 * G, window, 4, 0.0, 1024, size, None)
            assert e.value.code == A.HYB_ECUDA


def _delta(A, state=None, **kw):
    st = dict(state=256, n_slots=4, n_k_heads=2, n_v_heads=4, key_dim=64, value_dim=128)
    st.update(state or {})
    a = dict(q=256, q_stride=128, k=256, k_stride=128, v=256, v_stride=512, g=256, beta=256, out=256, out_stride=512, cu_new=64,
             slots=None, batch=2, n_new=2, max_new=1, scale=0.0, status=None, stream=None)
    a.update(kw)
    return A.hyb_attn_delta_run(A.hyb_attn_delta_state(**st), **a)


@pytest.mark.parametrize("state,kw", [(s, {}) for s in (dict(state=None), dict(state=8), dict(n_slots=0), dict(n_slots=1),
                                                        dict(n_k_heads=0), dict(n_k_heads=3), dict(key_dim=96),
                                                        dict(value_dim=32))] +
                         [({}, k) for k in (dict(q=None), dict(k=8), dict(v_stride=500), dict(v_stride=516), dict(q_stride=120),
                                            dict(g=None), dict(beta=2), dict(out=None), dict(out_stride=8), dict(cu_new=None),
                                            dict(slots=2), dict(batch=0), dict(max_new=0), dict(max_new=3), dict(n_new=-1),
                                            dict(scale=-1.0), dict(scale=float("nan")), dict(status=1))])
def test_delta_refuses(A, state, kw):
    with pytest.raises(A.HybAttnError) as e:
        _delta(A, state, **kw)
    assert e.value.code == A.HYB_EINVAL


def test_delta_no_rows_is_no_work(A):
    _delta(A, n_new=0, max_new=0, q=None, k=None, v=None, g=256, beta=256, out=None)


# ---- refusals of the classes -------------------------------------------------------------------------
def test_classes_need_a_gpu(A):
    import torch
    import hybrid_sparse_linear_decode_b200 as H
    codes = torch.zeros(4, 2, 16, 64, dtype=torch.int8)
    scales = torch.zeros(4, 2)
    if not torch.cuda.is_available():
        with pytest.raises(RuntimeError):
            H.PagedKVCache(4, 16, 2, 64)
        with pytest.raises(RuntimeError):
            H.GatedDeltaState(2, 1, 1, 64, 64)
    with pytest.raises(ValueError, match="CUDA"):
        H.PagedKVCache.from_tensors(codes, codes.clone(), scales, scales.clone())
    with pytest.raises(ValueError, match="codes are"):
        H.PagedKVCache.from_tensors(codes.float(), codes, scales, scales)
    with pytest.raises(ValueError, match="one shape"):
        H.PagedKVCache.from_tensors(codes, codes[:3], scales, scales)
    with pytest.raises(ValueError, match="scales"):
        H.PagedKVCache.from_tensors(codes, codes, scales[:3], scales)
    with pytest.raises(ValueError, match="CUDA"):
        H.GatedDeltaState.from_tensor(torch.zeros(2, 2, 64, 64), 1)
    with pytest.raises(ValueError, match="fp32"):
        H.GatedDeltaState.from_tensor(torch.zeros(2, 2, 64, 64, dtype=torch.float16), 1)


def test_calls_refuse_tensors_of_the_host(A):
    """The compiled calls check every tensor before anything is launched."""
    import torch
    from hybrid_sparse_linear_decode_b200._tensors import binding
    c, s = _cache(A), A.hyb_attn_delta_state(256, 4, 2, 4, 64, 128)
    at, st = ctypes.addressof(c), ctypes.addressof(s)
    row = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    ints = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="k has to be"):
        binding().paged_append(at, 0, 0, row, row, ints, ints[:2], ints[:2].view(2, 1), 1, None, False, None, None)
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        binding().paged_append(at, 0, 0, row.float(), row, ints, ints[:2], ints[:2].view(2, 1), 1, None, False, None, None)
    with pytest.raises(ValueError, match="q has to be"):
        binding().paged_attend(at, 0, 0, row, ints, ints[:2], ints[:2].view(2, 1), 1, 8, 0, 0, 0.0, None, False)
    with pytest.raises(ValueError, match="q has to be"):
        binding().delta_run(st, 0, 0, row, row, row, row, row, ints, 1, None, 0.0, None)


@pytest.mark.parametrize("type", [0, 1])
@pytest.mark.parametrize("head_dim,G", [(64, 1), (64, 16), (128, 4), (128, 8)])
def test_workspace_of_any_window_and_type_fits_the_workspace_asked_for(A, type, head_dim, G):
    """As above for both types, over more sequences, rows and lengths."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    rng = np.random.default_rng(head_dim + G)
    some = 0
    for _ in range(300):
        B, new, pages = (int(np.exp(rng.uniform(0, np.log(x)))) for x in (200, 3000, 3000))
        c = _cache(A, head_dim=head_dim)
        b = _batch(A, batch=B, n_new=B * new, max_new=new, table_stride=pages, max_len=16 * pages)
        size = A.hyb_attn_paged_workspace_size(c, b, 2 * G)
        some += size > 0
        for window in (0, 1, int(rng.integers(1, 16 * pages + 1)), int(rng.integers(1, 16 * pages + 1)), (1 << 31) - 1):
            with pytest.raises(A.HybAttnError) as e:
                A.hyb_attn_paged_attend(c, b, type, 256, 2 * G * head_dim, 512, 2 * G * head_dim, None, 2 * G, window, int(rng.integers(0, 100)), 0.0, 1024, size, None)
            assert e.value.code == A.HYB_ECUDA, (B, new, pages, window)
    assert some > 50


@pytest.mark.parametrize("scale", [1e-50, -1e-50, 5e-324])
def test_calls_refuse_a_scale_that_would_select_the_default(A, scale):
    """0 selects 1/sqrt(d); a scale that is 0 only in 32 bits is not one of them."""
    import torch
    from hybrid_sparse_linear_decode_b200._tensors import binding
    c, s = _cache(A), A.hyb_attn_delta_state(256, 4, 2, 4, 64, 128)
    row, ints = torch.zeros(2, 2, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="scale"):
        binding().paged_attend(ctypes.addressof(c), 0, 0, row, ints, ints[:2], ints[:2].view(2, 1), 1, 8, 0, 0, scale, None, False)
    with pytest.raises(ValueError, match="scale"):
        binding().delta_run(ctypes.addressof(s), 0, 0, row, row, row, row, row, ints, 1, None, scale, None)


# ---- the build -----------------------------------------------------------------------------------------
@pytest.mark.parametrize("what", [ImportError("no PyTorch"), RuntimeError("Python.h: no such file")])
def test_the_library_is_linked_without_the_binding(monkeypatch, tmp_path, what):
    """Without PyTorch or Python's headers only the calls that take tensors are missing."""
    from hybrid_sparse_linear_decode_b200 import build as B
    for name in ("LIB", "BINDING", "BUILD_DIR"):
        monkeypatch.setattr(B, name, str(tmp_path / name))
    monkeypatch.setattr(B, "SOURCES", ["api_delta.cu"])

    def fails(force):
        raise what

    monkeypatch.setattr(B, "compile_binding", fails)
    with pytest.raises(RuntimeError, match="is built"):
        B.build()
    assert (tmp_path / "LIB").exists() and not (tmp_path / "BINDING").exists()
