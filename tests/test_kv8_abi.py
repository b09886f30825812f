"""The 8-bit KV cache entry points without a GPU: refusals on the host, and pins of their oracle."""
import ctypes as C
import itertools

import numpy as np
import pytest
import torch

from block_diffusion_moe_dllm_b200 import binding as bd
from oracle import kv8_oracle as K8

FAKE = 0x10000  # never dereferenced: every call below fails validation first
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(bd.LIB_PATH):
        from block_diffusion_moe_dllm_b200 import build
        build.build()
    return bd.load()


# ------------------------------------------------------------------------------------------------ refusals
def _store(lib, src_pos=None, dst_rows=None, k=FAKE, codes=1 << 41, vc=5 << 40, **kw):
    f = dict(B=2, Hkv=4, d=128, n=32, cap_src=64, src_row=0, cap=96, dst_row=32, scale_len=32, dtype=bd.BF16,
             pos_stride=32)
    f.update(kw)
    d = bd.Kv8StoreDesc(**f)
    # arrays far enough apart; codes is the first output
    return lib.dllm_kv8_store(C.byref(d), k, 1 << 40, src_pos, dst_rows, codes, vc, 3 << 40, 4 << 40, None)


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), bd.ERR_INVALID_ARG), (dict(codes=None), bd.ERR_INVALID_ARG), (dict(dtype=7), bd.ERR_INVALID_ARG),
    (dict(B=0), bd.ERR_SHAPE), (dict(n=-1), bd.ERR_SHAPE), (dict(cap=31), bd.ERR_SHAPE),
    (dict(d=72), bd.ERR_UNSUPPORTED), (dict(d=144), bd.ERR_UNSUPPORTED), (dict(d=0), bd.ERR_UNSUPPORTED),
    (dict(scale_len=48), bd.ERR_UNSUPPORTED), (dict(scale_len=0), bd.ERR_UNSUPPORTED),
    (dict(src_row=33), bd.ERR_SHAPE), (dict(src_row=-1), bd.ERR_SHAPE), (dict(dst_row=16), bd.ERR_SHAPE),
    (dict(dst_row=96), bd.ERR_SHAPE), (dict(dst_row=-32), bd.ERR_SHAPE), (dict(src_pos=FAKE, pos_stride=31), bd.ERR_SHAPE),
    (dict(k=FAKE + 2), bd.ERR_ALIGN), (dict(codes=FAKE + 8), bd.ERR_ALIGN), (dict(codes=FAKE), bd.ERR_INVALID_ARG),
    (dict(vc=1 << 41), bd.ERR_INVALID_ARG), (dict(B=1 << 20, Hkv=1 << 12), bd.ERR_UNSUPPORTED)])
def test_store_refuses(lib, kw, code):
    assert _store(lib, **kw) == code
    assert "kv8_store" in lib.dllm_last_error().decode()


def _attn(lib, q=FAKE, codes=FAKE, own=(1 << 21, 1 << 22), out=1 << 23, ws=FAKE, ws_bytes=BIG, **kw):
    f = dict(B=2, Lq=32, Hq=16, Hkv=4, d=128, blk_len=32, P=256, cap=256, cap_own=32, scale_len=32, dtype=bd.BF16,
             scale=0.0)
    f.update(kw)
    d = bd.AttnKv8Desc(**f)
    return lib.dllm_block_attn_kv8(C.byref(d), q, codes, FAKE, FAKE, FAKE, None, own[0], own[1], out, None, ws, ws_bytes,
                                   None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), bd.ERR_INVALID_ARG), (dict(codes=None), bd.ERR_INVALID_ARG), (dict(out=None), bd.ERR_INVALID_ARG),
    (dict(own=(FAKE, None)), bd.ERR_INVALID_ARG), (dict(out=FAKE + 64), bd.ERR_INVALID_ARG),
    (dict(dtype=2), bd.ERR_INVALID_ARG), (dict(Hq=18), bd.ERR_SHAPE), (dict(Lq=0), bd.ERR_SHAPE),
    (dict(P=-1), bd.ERR_SHAPE), (dict(cap=255), bd.ERR_SHAPE), (dict(cap_own=31), bd.ERR_SHAPE),
    (dict(blk_len=0), bd.ERR_SHAPE), (dict(d=64), bd.ERR_UNSUPPORTED), (dict(scale_len=8), bd.ERR_UNSUPPORTED),
    (dict(d=72, dtype=bd.F32), bd.ERR_UNSUPPORTED), (dict(q=FAKE + 4), bd.ERR_ALIGN), (dict(codes=FAKE + 1), bd.ERR_ALIGN),
    (dict(own=(FAKE + 8, FAKE)), bd.ERR_ALIGN), (dict(ws=None), bd.ERR_WORKSPACE), (dict(ws=FAKE + 16), bd.ERR_WORKSPACE),
    (dict(ws_bytes=64), bd.ERR_WORKSPACE), (dict(Lq=1 << 24, cap_own=1 << 24), bd.ERR_UNSUPPORTED),
    (dict(B=1 << 22), bd.ERR_UNSUPPORTED)])
def test_block_attn_kv8_refuses(lib, kw, code):
    assert _attn(lib, **kw) == code


def _mass(lib, q=FAKE, lse=FAKE, mass_in=1 << 24, mass_out=1 << 25, ws=FAKE, **kw):
    f = dict(B=2, Lq=32, Hq=16, Hkv=4, d=128, P=256, cap=256, scale_len=32, dtype=bd.BF16, scale=0.0, decay=1.0)
    f.update(kw)
    d = bd.AttnMassDesc(**f)
    return lib.dllm_attn_mass_kv8(C.byref(d), q, FAKE, FAKE, None, lse, mass_in, mass_out, ws, BIG, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), bd.ERR_INVALID_ARG), (dict(lse=None), bd.ERR_INVALID_ARG), (dict(mass_out=None), bd.ERR_INVALID_ARG),
    (dict(mass_in=(1 << 25) + 4), bd.ERR_INVALID_ARG), (dict(Hkv=3), bd.ERR_SHAPE), (dict(cap=10), bd.ERR_SHAPE),
    (dict(d=96), bd.ERR_UNSUPPORTED), (dict(q=FAKE + 2), bd.ERR_ALIGN), (dict(ws=None), bd.ERR_WORKSPACE)])
def test_attn_mass_kv8_refuses(lib, kw, code):
    assert _mass(lib, **kw) == code


def _evict(lib, ptrs=None, ws=FAKE, pos=None, **kw):
    f = dict(B=2, Hkv=4, d=128, P=256, cap=256, n_keep=64, cap_out=64, scale_len=32, n_first=4, n_last=16, per_head=0)
    f.update(kw)
    d = bd.Kv8EvictDesc(**f)
    p = [(i + 1) << 24 for i in range(12)]
    for i, x in (ptrs or {}).items():
        p[i] = x
    return lib.dllm_kv8_evict(C.byref(d), *p[:5], None, pos, *p[5:], ws, BIG, None)


@pytest.mark.parametrize("kw,code", [
    (dict(ptrs={0: None}), bd.ERR_INVALID_ARG), (dict(ptrs={11: None}), bd.ERR_INVALID_ARG),
    (dict(ptrs={5: 1 << 24}), bd.ERR_INVALID_ARG),                      # in place: k_out on k_codes
    (dict(ptrs={9: (5 << 24) + 256}), bd.ERR_INVALID_ARG),              # mass_out inside mass
    (dict(ptrs={6: 6 << 24}), bd.ERR_INVALID_ARG),                      # v_out on k_out
    (dict(n_keep=0), bd.ERR_SHAPE), (dict(n_keep=65), bd.ERR_SHAPE), (dict(n_first=50, n_last=15), bd.ERR_INVALID_ARG),
    (dict(n_first=-1), bd.ERR_INVALID_ARG), (dict(cap=100), bd.ERR_SHAPE), (dict(scale_len=20), bd.ERR_UNSUPPORTED),
    (dict(d=100), bd.ERR_UNSUPPORTED), (dict(ptrs={6: (7 << 24) + 8}), bd.ERR_ALIGN), (dict(ws=None), bd.ERR_WORKSPACE)])
def test_kv8_evict_refuses(lib, kw, code):
    assert _evict(lib, **kw) == code


def test_workspace_sizes_of_refused_shapes_are_zero_or_plain(lib):
    size = lib.dllm_block_attn_kv8_workspace_size
    d = bd.AttnKv8Desc(1, 32, 16, 0, 128, 32, 256, 256, 32, 32, bd.BF16, 0.0)
    assert size(C.byref(d)) == 0 and size(None) == 0
    assert lib.dllm_kv8_evict_workspace_size(None) == 0 and lib.dllm_attn_mass_kv8_workspace_size(None) == 0
    e = bd.Kv8EvictDesc(2, 4, 128, 256, 256, 64, 64, 32, 0, 0, 0)
    f = bd.Kv8EvictDesc(2, 4, 128, 256, 256, 64, 64, 32, 0, 0, 1)
    assert lib.dllm_kv8_evict_workspace_size(C.byref(f)) > lib.dllm_kv8_evict_workspace_size(C.byref(e)) > 0


@pytest.mark.parametrize("at", ["out=k_own", "out=v_own", "out=codes", "out=k_scale", "out=lens", "lse=out", "lse=q",
                                "lse=v_scale"])
def test_block_attn_kv8_refuses_outputs_on_other_arrays(lib, at):
    p = dict(q=1 << 30, codes=2 << 30, vc=3 << 30, k_scale=4 << 30, v_scale=5 << 30, lens=6 << 30, k_own=7 << 30,
             v_own=8 << 30, out=9 << 30, lse=10 << 30)
    which, on = at.split("=")
    d = bd.AttnKv8Desc(2, 32, 16, 4, 128, 32, 256, 256, 32, 32, bd.BF16, 0.0)

    def call(ws):
        return lib.dllm_block_attn_kv8(C.byref(d), *p.values(), ws, BIG, None)

    assert call(None) == bd.ERR_WORKSPACE                    # these arrays are fine
    # the last 16 bytes that the call reads of the other array (one row tensor each of 2 batch rows)
    span = dict(q=2 * 32 * 16 * 128 * 2, codes=2 * 4 * 256 * 128, k_scale=2 * 4 * 8 * 4, v_scale=2 * 4 * 8 * 4, lens=8,
                k_own=2 * 4 * 32 * 128 * 2, v_own=2 * 4 * 32 * 128 * 2, out=2 * 32 * 16 * 128 * 2)[on]
    first = p[on]
    p[which] = first + (span - 1) // 16 * 16
    assert call(None) == bd.ERR_INVALID_ARG
    p[which] = first + (span + 15) // 16 * 16
    assert call(None) == bd.ERR_WORKSPACE


@pytest.mark.parametrize("on,span", [(1, 2 * 32 * 16 * 128 * 2), (2, 2 * 4 * 256 * 128), (3, 2 * 4 * 8 * 4), (4, 8),
                                     (5, 2 * 32 * 16 * 4)])
def test_attn_mass_kv8_refuses_its_output_on_other_arrays(lib, on, span):
    d = bd.AttnMassDesc(2, 32, 16, 4, 128, 256, 256, 32, bd.BF16, 0.0, 1.0)
    p = [i << 30 for i in range(1, 6)]                       # q, codes, k_scale, lengths, lse
    for off, code in ((span - 4, bd.ERR_INVALID_ARG), (span, bd.ERR_WORKSPACE)):
        m = (on << 30) + off
        assert lib.dllm_attn_mass_kv8(C.byref(d), *p, m, m, None, BIG, None) == code


def test_store_refuses_an_output_on_its_row_list(lib):
    assert _store(lib, dst_rows=(1 << 41) + 64) == bd.ERR_INVALID_ARG


def test_workspace_size_of_more_rows_than_a_call_takes_is_zero(lib):
    # rows per kv head of 2^32 and beyond, at which a 32-bit product is zero or negative
    for Lq, Hq, B, P in ((1 << 16, 1 << 16, 1, 256), (1 << 17, 1 << 14, 1, 256), (32, 16, 1 << 30, 256), (1, 1, 1 << 24, 1 << 30)):
        for dt in (bd.BF16, bd.F32):
            d = bd.AttnKv8Desc(B, Lq, Hq, 1, 128, 32, P, P, 32, 32, dt, 0.0)
            assert lib.dllm_block_attn_kv8_workspace_size(C.byref(d)) == 0


def test_a_workspace_is_taken_on_the_calls_stream(monkeypatch):
    """A workspace that a call takes or grows is filled on the call's stream, which also orders who gets it next."""
    seen = []

    class On:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            seen.append(self.stream)

        def __exit__(self, *_):
            seen.append("left")

    monkeypatch.setattr(torch.cuda, "stream", On)
    ws = bd._stream_workspace(None, 1000, "cpu", "side")
    assert seen == ["side", "left"] and ws.nbytes == 1000
    assert bd._stream_workspace(ws, 1000, "cpu", "side") is ws and len(seen) == 2
    assert bd._stream_workspace(ws, 5000, "cpu", "other").nbytes == 5000 and seen[2:] == ["other", "left"]


# ------------------------------------------------------------------------------------------------ oracle pins
def test_e4m3_values_and_rounding_match_torch():
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(K8.e4m3_values(), want, equal_nan=True)
    g = np.random.default_rng(0)
    finite = np.sort(want[np.isfinite(want)])
    x = np.concatenate([g.normal(0, 1, 4000) * 2.0 ** g.integers(-12, 9, 4000), (finite[1:] + finite[:-1]) / 2, finite])
    x = x[np.abs(x) <= 448].astype(np.float32)
    assert np.array_equal(K8.round_e4m3(x), torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy())
    assert K8.round_e4m3(np.inf) == 448 and K8.round_e4m3(-500.0) == -448 and np.isnan(K8.round_e4m3(np.nan))


@pytest.mark.parametrize("amax,k", [(448.0, 0), (448.1, 1), (224.0, -1), (1.75, -8), (1.7500001, -7), (1e-30, -64),
                                    (3.3e38, 120), (0.0, -64)])
def test_run_scale(amax, k):
    assert K8.run_scale(np.array([[amax, -amax / 3]])) == 2.0 ** k


def test_attention_pins():
    """No cache rounding: equals library attention on the concatenated keys; a row without keys is zero."""
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((1, 4, 2, 16), (1, 2, 9, 16), (1, 2, 9, 16)))
    want = torch.nn.functional.scaled_dot_product_attention(q.transpose(1, 2), k, v).transpose(1, 2)
    o, lse, _, _ = K8.attention(q.numpy(), k[:, :, :5].numpy(), v[:, :, :5].numpy(), [5], k[:, :, 5:].numpy(),
                                v[:, :, 5:].numpy(), 4)
    assert np.allclose(o, want.numpy(), atol=1e-12)
    m = K8.mass(q.numpy(), k.numpy(), [9], lse, None, np.zeros((1, 2, 9)))
    assert np.allclose(m.sum(-1), 4.0)                       # every query spends weight 1 per head
    o, lse, _, _ = K8.attention(q.numpy(), k.numpy(), v.numpy(), [0], None, None, 4)
    assert not o.any() and np.all(lse == -np.inf)


def test_select_brute_force():
    g = np.random.default_rng(3)
    for n, keep, first, last in itertools.product((1, 5, 8), (1, 3, 8), (0, 1), (0, 1)):
        if first + last > keep:
            continue
        m = g.integers(0, 3, (2, n)).astype(np.float64)       # many ties
        rows = K8.select(m, n, keep, first, last)
        assert len(rows) == min(n, keep) and list(rows) == sorted(set(rows))
        must = set(range(min(first, n))) | set(range(max(0, n - last), n))
        assert must <= set(rows)
        t = m.sum(0)
        for j in set(range(n)) - set(rows):
            for i in set(rows) - must:
                assert t[i] > t[j] or (t[i] == t[j] and i < j)
