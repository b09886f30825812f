"""The 8-bit KV cache entry points without a GPU: which arrays may lie beside or between others, and where tensors may be."""
import ctypes as C

import pytest

from block_diffusion_moe_dllm_b200 import binding as bd

GB = 1 << 30


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(bd.LIB_PATH):
        from block_diffusion_moe_dllm_b200 import build
        build.build()
    return bd.load()


# Addresses are never dereferenced: a call that passes the checks under test is refused by one after them. The store has none,
# so what it accepts is not called here: its n = 0 form returns after the checks.
def _store(lib, n=32, src_pos=None, pos_stride=40, **p):
    a = dict(k=1 * GB, v=2 * GB, kc=3 * GB, vc=4 * GB, ks=5 * GB, vs=6 * GB)
    a.update(p)
    d = bd.Kv8StoreDesc(B=2, Hkv=4, d=128, n=n, cap_src=64, src_row=0, cap=96, dst_row=32, scale_len=32, dtype=bd.BF16,
                        pos_stride=pos_stride)
    return lib.dllm_kv8_store(C.byref(d), a["k"], a["v"], src_pos, None, a["kc"], a["vc"], a["ks"], a["vs"], None)


@pytest.mark.parametrize("out", ["kc", "vc", "ks", "vs"])
def test_store_refuses_an_output_on_its_position_list(lib, out):
    at = 9 * GB
    # the list's last entry: batch row 1, token 31
    assert _store(lib, src_pos=at, **{out: at + (1 * 40 + 31) * 4 // 16 * 16}) == bd.ERR_INVALID_ARG
    assert "kv8_store" in lib.dllm_last_error().decode()
    assert _store(lib, src_pos=at, **{out: at}) == bd.ERR_INVALID_ARG
    assert _store(lib, n=0, src_pos=at, **{out: at}) == bd.OK                # nothing is read or written


def _attn(lib, ws, **p):
    a = dict(q=1 * GB, kc=2 * GB, vc=3 * GB, ks=4 * GB, vs=5 * GB, lens=6 * GB, ko=7 * GB, vo=8 * GB, out=9 * GB, lse=10 * GB)
    a.update(p)
    d = bd.AttnKv8Desc(2, 32, 16, 4, 128, 32, 256, 256, 32, 32, bd.BF16, 0.0)
    return lib.dllm_block_attn_kv8(C.byref(d), *a.values(), ws, 1 << 40, None)


@pytest.mark.parametrize("on", ["q", "kc", "vc", "ks", "vs", "lens", "ko", "vo", "out", "lse"])
def test_block_attn_kv8_refuses_its_workspace_on_other_arrays(lib, on):
    d = bd.AttnKv8Desc(2, 32, 16, 4, 128, 32, 256, 256, 32, 32, bd.BF16, 0.0)
    ws = 64 * GB
    last = ws + lib.dllm_block_attn_kv8_workspace_size(C.byref(d)) - 256
    for at in (ws, last):
        assert _attn(lib, ws, **{on: at}) == bd.ERR_INVALID_ARG
        assert "workspace" in lib.dllm_last_error().decode()


@pytest.mark.parametrize("on", range(6))
def test_attn_mass_kv8_refuses_its_workspace_on_other_arrays(lib, on):
    d = bd.AttnMassDesc(2, 32, 16, 4, 128, 256, 256, 32, bd.BF16, 0.0, 1.0)
    p = [i * GB for i in range(1, 7)]                       # q, codes, k_scale, lengths, lse, mass
    ws = 64 * GB
    p[on] = ws
    assert lib.dllm_attn_mass_kv8(C.byref(d), *p, p[5], ws, 1 << 40, None) == bd.ERR_INVALID_ARG
    assert "workspace" in lib.dllm_last_error().decode()


@pytest.mark.parametrize("on", range(14))
def test_kv8_evict_refuses_its_workspace_on_other_arrays(lib, on):
    d = bd.Kv8EvictDesc(2, 4, 128, 256, 256, 64, 64, 32, 4, 16, 0)
    p = [i * GB for i in range(1, 15)]                      # inputs, lengths, positions, outputs
    ws = 64 * GB
    p[on] = ws
    assert lib.dllm_kv8_evict(C.byref(d), *p, ws, 1 << 40, None) == bd.ERR_INVALID_ARG
    assert "workspace" in lib.dllm_last_error().decode()


def test_parts_of_longer_arrays_may_lie_side_by_side(lib):
    """Two caches of 1024 rows in one allocation of 2048, the eviction from the tail of the first (rows 512 on, as far apart
    as the whole) to the second: the part's last head ends where the second begins."""
    B, Hkv, d, cap, r0, S, keep = 1, 2, 128, 1024, 512, 32, 256
    P = cap - r0
    e = bd.Kv8EvictDesc(B, Hkv, d, P, cap, keep, cap, S, 0, 0, 0)
    code, scale, mass = Hkv * cap * d, Hkv * cap // S * 4, Hkv * cap * 4

    def call(shift, ws):
        k, v, ks, vs, m = 1 * GB, 2 * GB, 3 * GB, 4 * GB, 5 * GB
        return lib.dllm_kv8_evict(C.byref(e), k + r0 * d, v + r0 * d, ks + r0 // S * 4, vs + r0 // S * 4, m + r0 * 4, None,
                                  None, k + code - shift, v + code, ks + scale, vs + scale, m + mass, 6 * GB, 7 * GB, ws,
                                  1 << 40, None)

    assert call(0, None) == bd.ERR_WORKSPACE                # passed the arrays' check
    assert call(16, None) == bd.ERR_INVALID_ARG             # into the part's last row
    # the weights of such a part, in an accumulator that ends where the next one begins
    a = bd.AttnMassDesc(B, 32, 4, Hkv, d, P, cap, S, bd.BF16, 0.0, 1.0)
    for off, code_ in ((mass, bd.ERR_WORKSPACE), (mass - 4, bd.ERR_INVALID_ARG)):
        assert lib.dllm_attn_mass_kv8(C.byref(a), 1 * GB, 2 * GB, 3 * GB, None, 4 * GB, 5 * GB + off, 5 * GB + r0 * 4, None,
                                      1 << 40, None) == code_


# ------------------------------------------------------------------------------------------------ the binding
class On:
    """A tensor's place, as the binding looks at it."""

    def __init__(self, device, nbytes=1 << 20):
        self.device, self.nbytes, self.addr, self.buf = device, nbytes, 256, self

    def get_device(self):
        return self.device

    def data_ptr(self):
        return 256


@pytest.mark.parametrize("where", [-1, 1])
def test_each_tensor_has_to_be_on_the_current_device(monkeypatch, where):
    """Every tensor of every call, one at a time on the host (-1) or on another device, is refused before the library is
    called."""
    import torch
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    sizes = dict(B=1, Hkv=1, d=128, cap=16, scale_len=16)
    q = dict(Lq=1, Hq=1, P=16, dtype=bd.BF16)
    calls = [(bd.kv8_store, ["k", "v", "k_codes", "v_codes", "k_scale", "v_scale", "src_pos", "dst_rows"],
              dict(sizes, n=16, cap_src=16, dtype=bd.BF16)),
             (bd.block_attn_kv8, ["q", "k_codes", "v_codes", "k_scale", "v_scale", "out", "prefix_len", "k_own", "v_own", "lse",
                                  "ws"], dict(sizes, **q, blk_len=1, cap_own=1)),
             (bd.attn_mass_kv8, ["q", "k_codes", "k_scale", "lse", "mass_in", "mass_out", "prefix_len", "ws"],
              dict(sizes, **q)),
             (bd.kv8_evict, ["k_codes", "v_codes", "k_scale", "v_scale", "mass", "k_out", "v_out", "k_scale_out",
                             "v_scale_out", "mass_out", "keep_pos", "len_out", "prefix_len", "pos", "ws"],
              dict(sizes, P=16, n_keep=8, cap_out=8))]
    for call, names, rest in calls:
        for bad in names:
            tensors = {n: On(where if n == bad else 0, 1 << 30) for n in names}
            with pytest.raises(bd.DllmError) as e:
                call(**tensors, **rest)
            assert e.value.code == bd.ERR_INVALID_ARG and "current device" in str(e.value), (call.__name__, bad)


def test_stream_handle_without_the_short_way(monkeypatch):
    import torch

    class Stream:
        cuda_stream = 77

    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream)
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    assert bd._raw_stream(0) == 77
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 1000 + dev, raising=False)
    assert bd._raw_stream(3) == 1003
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    assert bd._launch_args(Stream, None, On(0)) == [None, 256, 77] and bd._launch_args(None) == [1000]
